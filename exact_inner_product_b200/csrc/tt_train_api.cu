// tt_train_api.cu - the C ABI of the training-step operators: argument
// validation and launches. Conventions and errors as in tt_api.cu.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "../../include/tt.h"
#include "tt_internal.h"

#define TT_CUDA(call, what)                                \
    do {                                                   \
        const cudaError_t _e = (call);                     \
        if (_e != cudaSuccess) return cuda_fail(_e, what); \
    } while (0)

namespace tt {
namespace {

size_t elem_bytes(int dtype) { return dtype == TT_F32 ? 4 : 2; }

bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
    if (a == nullptr || b == nullptr || a_bytes == 0 || b_bytes == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

// Device pointers of a call, one query per allocation: what lies in the
// allocation of the pointer checked last needs none (a list of a few hundred
// gradients is mostly views into few of them).
class DeviceCheck {
    uintptr_t lo = 0, hi = 0;
    typedef CUresult (*RangeFn)(CUdeviceptr*, size_t*, CUdeviceptr);
    static RangeFn range_fn() {
        static const RangeFn fn = [] {
            void* p = nullptr;
            cudaDriverEntryPointQueryResult q;
            const cudaError_t e = cudaGetDriverEntryPoint("cuMemGetAddressRange", &p, cudaEnableDefault, &q);
            return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<RangeFn>(p) : nullptr;
        }();
        return fn;
    }

public:
    tt_status operator()(const void* p, const char* name) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        if (p == nullptr || (at >= lo && at < hi)) return TT_OK;
        const tt_status st = check_device_ptr(p, name);
        if (st != TT_OK) return st;
        CUdeviceptr base = 0;
        size_t size = 0;
        if (range_fn() != nullptr && range_fn()(&base, &size, (CUdeviceptr)at) == CUDA_SUCCESS) {
            lo = (uintptr_t)base;
            hi = lo + size;
        }
        return TT_OK;
    }
};

// The buffers of a call. Outputs may overlap nothing; inputs may overlap
// inputs. Null buffers are skipped.
struct Buffers {
    struct One {
        const void* p;
        size_t bytes;
        const char* name;
        bool out;
    };
    One list[20];
    int count = 0;
    void add(const void* p, size_t bytes, const char* name, bool out) {
        if (p != nullptr) list[count++] = {p, bytes, name, out};
    }
    void in(const void* p, size_t bytes, const char* name) { add(p, bytes, name, false); }
    void out(const void* p, size_t bytes, const char* name) { add(p, bytes, name, true); }
    // host-side check, then the device pointers
    tt_status check() const {
        for (int i = 0; i < count; ++i)
            for (int j = 0; j < i; ++j)
                if ((list[i].out || list[j].out) && overlap(list[i].p, list[i].bytes, list[j].p, list[j].bytes)) {
                    char msg[160];
                    snprintf(msg, sizeof msg, "%s overlaps %s", list[i].name, list[j].name);
                    set_last_error_message(msg);
                    return TT_ERR_INVALID_ARG;
                }
        DeviceCheck device;
        for (int i = 0; i < count; ++i) {
            const tt_status st = device(list[i].p, list[i].name);
            if (st != TT_OK) return st;
        }
        return TT_OK;
    }
};

tt_status check_workspace(const void* workspace, size_t have, size_t need) {
    if (workspace == nullptr || !aligned(workspace, 256)) return TT_ERR_INVALID_ARG;
    if (have < need) {
        char msg[96];
        snprintf(msg, sizeof msg, "workspace of %zu bytes, need %zu", have, need);
        set_last_error_message(msg);
        return TT_ERR_INVALID_ARG;
    }
    return TT_OK;
}

tt_status check_rows(int64_t n, int32_t d) {
    if (n < 0 || d <= 0) return TT_ERR_INVALID_ARG;
    if (n > TT_MAX_N || d > TT_MAX_WIDTH) return TT_ERR_UNSUPPORTED;
    return TT_OK;
}

tt_status check_clip_list(int32_t count, const int64_t* n, const int32_t* dtypes) {
    if (count < 0 || (count > 0 && (n == nullptr || dtypes == nullptr))) return TT_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        if (!valid_dtype(dtypes[i]) || n[i] < 0) return TT_ERR_INVALID_ARG;
        if (n[i] >= (int64_t)1 << 42) return TT_ERR_UNSUPPORTED;
    }
    return TT_OK;
}

// No output overlaps another output, or an input other than its own.
tt_status check_clip_overlap(const ClipList& l) {
    struct Range {
        uintptr_t lo, hi;
        bool out;
        bool operator<(const Range& o) const { return lo < o.lo; }
    };
    Range* r = static_cast<Range*>(malloc(sizeof(Range) * 2 * (size_t)(l.count > 0 ? l.count : 1)));
    if (r == nullptr) return TT_ERR_NO_MEMORY;
    int k = 0;
    for (int i = 0; i < l.count; ++i) {
        if (l.n[i] == 0) continue;
        const size_t bytes = (size_t)l.n[i] * elem_bytes(l.dtype[i]);
        const uintptr_t in = reinterpret_cast<uintptr_t>(l.in[i]), out = reinterpret_cast<uintptr_t>(l.out[i]);
        r[k++] = {out, out + bytes, true};
        if (in != out) r[k++] = {in, in + bytes, false};
    }
    if (!std::is_sorted(r, r + k)) std::sort(r, r + k);
    uintptr_t out_end = 0, in_end = 0;
    bool bad = false;
    for (int i = 0; i < k && !bad; ++i) {
        bad = r[i].lo < out_end || (r[i].out && r[i].lo < in_end);
        uintptr_t& end = r[i].out ? out_end : in_end;
        if (r[i].hi > end) end = r[i].hi;
    }
    free(r);
    if (bad) set_last_error_message("an output overlaps another tensor of the call");
    return bad ? TT_ERR_INVALID_ARG : TT_OK;
}

tt_status clip(const ClipList& l, bool scale, float max_norm, float* norm, void* workspace, size_t workspace_bytes,
               void* stream) {
    tt_status st = check_clip_list(l.count, l.n, l.dtype);
    if (st != TT_OK) return st;
    if (l.count > 0 && (l.in == nullptr || l.out == nullptr)) return TT_ERR_INVALID_ARG;
    if (!(max_norm >= 0.0f) || norm == nullptr || !aligned(norm, 4)) return TT_ERR_INVALID_ARG;
    for (int i = 0; i < l.count; ++i) {
        if (l.n[i] == 0) continue;
        if (l.in[i] == nullptr || !aligned(l.in[i], elem_bytes(l.dtype[i]))) return TT_ERR_INVALID_ARG;
        if (scale && (l.out[i] == nullptr || !aligned(l.out[i], elem_bytes(l.dtype[i])))) return TT_ERR_INVALID_ARG;
    }
    const int sms = sm_count_current();
    const size_t need = clip_workspace_bytes(l, sms);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != TT_OK) return st;
    if (scale && (st = check_clip_overlap(l)) != TT_OK) return st;
    DeviceCheck grads, outs;
    for (int i = 0; i < l.count; ++i) {
        if (l.n[i] == 0) continue;
        const size_t bytes = (size_t)l.n[i] * elem_bytes(l.dtype[i]);
        if (overlap(l.in[i], bytes, norm, 4) || overlap(l.in[i], bytes, workspace, need) ||
            (scale && (overlap(l.out[i], bytes, norm, 4) || overlap(l.out[i], bytes, workspace, need)))) {
            set_last_error_message("norm or workspace overlaps a tensor");
            return TT_ERR_INVALID_ARG;
        }
        if ((st = grads(l.in[i], "grads")) != TT_OK) return st;
        if (scale && l.out[i] != l.in[i] && (st = outs(l.out[i], "out")) != TT_OK) return st;
    }
    if (overlap(norm, 4, workspace, need)) return TT_ERR_INVALID_ARG;
    if ((st = check_device_ptr(norm, "norm")) != TT_OK) return st;
    if ((st = check_device_ptr(workspace, "workspace")) != TT_OK) return st;
    const cudaError_t e = launch_clip(l, scale, max_norm, norm, static_cast<double*>(workspace),
                                      static_cast<cudaStream_t>(stream), sms);
    return e == cudaSuccess ? TT_OK : cuda_fail(e, "gradient norm");
}

tt_status check_embedding(int64_t rows, int32_t d, int32_t id_bytes, int64_t m, float scale) {
    tt_status st = check_rows(rows, d);
    if (st != TT_OK) return st;
    if ((st = check_rows(m, d)) != TT_OK) return st;
    if ((id_bytes != 4 && id_bytes != 8) || !isfinite(scale)) return TT_ERR_INVALID_ARG;
    return TT_OK;
}

tt_status embedding_grad(const EmbeddingGrad& g, bool by_row, size_t workspace_bytes, void* stream) {
    tt_status st = check_embedding(g.rows, g.d, g.id_bytes, g.m, g.scale);
    if (st != TT_OK) return st;
    if (!valid_dtype(g.grad_dtype) || !valid_dtype(g.out_dtype)) return TT_ERR_INVALID_ARG;
    if (!aligned(g.ids, g.id_bytes) || !aligned(g.grad, 16) || !aligned(g.out, 16) || !aligned(g.out_ids, g.id_bytes) ||
        !aligned(g.count, 4))
        return TT_ERR_INVALID_ARG;
    if (g.m > 0 && (g.ids == nullptr || g.grad == nullptr)) return TT_ERR_INVALID_ARG;
    if (by_row ? (g.count == nullptr || (g.m > 0 && (g.out == nullptr || g.out_ids == nullptr)))
               : (g.rows > 0 && g.out == nullptr))
        return TT_ERR_INVALID_ARG;
    const size_t need = embedding_grad_bytes(g.m, g.rows, g.d);
    if ((st = check_workspace(g.workspace, workspace_bytes, need)) != TT_OK) return st;
    Buffers b;
    b.in(g.ids, (size_t)g.m * g.id_bytes, "ids");
    b.in(g.grad, (size_t)g.m * g.d * elem_bytes(g.grad_dtype), "grad");
    b.out(g.out, (size_t)(by_row ? g.m : g.rows) * g.d * elem_bytes(g.out_dtype), by_row ? "out_rows" : "grad_table");
    b.out(g.out_ids, (size_t)g.m * g.id_bytes, "out_ids");
    b.out(g.count, sizeof(int32_t), "count");
    b.out(g.workspace, need, "workspace");
    if ((st = b.check()) != TT_OK) return st;
    const cudaError_t e = launch_embedding_grad(g, by_row, static_cast<cudaStream_t>(stream), sm_count_current());
    return e == cudaSuccess ? TT_OK : cuda_fail(e, "embedding gradient");
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" {

tt_status tt_layernorm(const void* x, tt_dtype dtype, int64_t n, int32_t d, const void* w, const void* bias,
                       tt_dtype w_dtype, float eps, void* y, float* mean, float* rstd, void* stream) {
    tt_status st = check_rows(n, d);
    if (st != TT_OK) return st;
    if (!valid_dtype(dtype) || !valid_dtype(w_dtype)) return TT_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !isfinite(eps)) return TT_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return TT_ERR_INVALID_ARG;
    if (n == 0) return TT_OK;
    if (x == nullptr || y == nullptr) return TT_ERR_INVALID_ARG;
    const size_t row_bytes = (size_t)n * d * elem_bytes(dtype), w_bytes = d * elem_bytes(w_dtype);
    Buffers b;
    b.in(x, row_bytes, "x");
    b.in(w, w_bytes, "w");
    b.in(bias, w_bytes, "bias");
    b.out(y, row_bytes, "y");
    b.out(mean, n * sizeof(float), "mean");
    b.out(rstd, n * sizeof(float), "rstd");
    if ((st = b.check()) != TT_OK) return st;
    const cudaError_t e = launch_layernorm(x, dtype, n, d, w, bias, w_dtype, eps, y, mean, rstd,
                                           static_cast<cudaStream_t>(stream), sm_count_current());
    return e == cudaSuccess ? TT_OK : cuda_fail(e, "layer norm");
}

tt_status tt_layernorm_grad_workspace(int64_t n, int32_t d, size_t* bytes) {
    if (bytes == nullptr) return TT_ERR_INVALID_ARG;
    const tt_status st = check_rows(n, d);
    if (st != TT_OK) return st;
    *bytes = layernorm_grad_bytes(n, d, sm_count_current());
    return TT_OK;
}

tt_status tt_layernorm_grad(const void* grad_y, const void* x, tt_dtype dtype, int64_t n, int32_t d, const void* w,
                            tt_dtype w_dtype, const float* mean, const float* rstd, void* grad_x, float* grad_w,
                            float* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
    tt_status st = check_rows(n, d);
    if (st != TT_OK) return st;
    if (!valid_dtype(dtype) || !valid_dtype(w_dtype)) return TT_ERR_INVALID_ARG;
    if (!aligned(grad_y, 16) || !aligned(x, 16) || !aligned(grad_x, 16) || !aligned(w, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(grad_w, 4) || !aligned(grad_bias, 4))
        return TT_ERR_INVALID_ARG;
    if (n > 0 && (grad_y == nullptr || x == nullptr || mean == nullptr || rstd == nullptr)) return TT_ERR_INVALID_ARG;
    const int sms = sm_count_current();
    const size_t need = layernorm_grad_bytes(n, d, sms);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != TT_OK) return st;
    const size_t row_bytes = (size_t)n * d * elem_bytes(dtype);
    Buffers b;
    b.in(grad_y, row_bytes, "grad_y");
    b.in(x, row_bytes, "x");
    b.in(w, d * elem_bytes(w_dtype), "w");
    b.in(mean, n * sizeof(float), "mean");
    b.in(rstd, n * sizeof(float), "rstd");
    b.out(grad_x, row_bytes, "grad_x");
    b.out(grad_w, d * sizeof(float), "grad_w");
    b.out(grad_bias, d * sizeof(float), "grad_bias");
    b.out(workspace, need, "workspace");
    if ((st = b.check()) != TT_OK) return st;
    const cudaError_t e =
        launch_layernorm_grad(grad_y, x, dtype, n, d, w, w_dtype, mean, rstd, grad_x, grad_w, grad_bias,
                              static_cast<float*>(workspace), static_cast<cudaStream_t>(stream), sms);
    return e == cudaSuccess ? TT_OK : cuda_fail(e, "layer norm gradient");
}

tt_status tt_normalize_grad(const void* grad_y, tt_dtype g_dtype, const void* x, tt_dtype dtype, int64_t n, int32_t d,
                            void* grad_x, void* stream) {
    if (n < 0 || d <= 0) return TT_ERR_INVALID_ARG;
    if (n > TT_MAX_N || d % 16 != 0 || d > TT_MAX_D) return TT_ERR_UNSUPPORTED;
    if (!valid_dtype(dtype) || !valid_dtype(g_dtype)) return TT_ERR_INVALID_ARG;
    if (!aligned(grad_y, 16) || !aligned(x, 16) || !aligned(grad_x, 16)) return TT_ERR_INVALID_ARG;
    if (n == 0) return TT_OK;
    if (grad_y == nullptr || x == nullptr || grad_x == nullptr) return TT_ERR_INVALID_ARG;
    const size_t elems = (size_t)n * d;
    Buffers b;
    b.in(grad_y, elems * elem_bytes(g_dtype), "grad_y");
    b.in(x, elems * elem_bytes(dtype), "x");
    b.out(grad_x, elems * elem_bytes(dtype), "grad_x");
    tt_status st = b.check();
    if (st != TT_OK) return st;
    const cudaError_t e = launch_normalize_grad(grad_y, g_dtype, x, dtype, n, d, grad_x,
                                                static_cast<cudaStream_t>(stream), sm_count_current());
    return e == cudaSuccess ? TT_OK : cuda_fail(e, "normalisation gradient");
}

tt_status tt_clip_grad_norm_workspace(int32_t count, const int64_t* n, const int32_t* dtypes, size_t* bytes) {
    if (bytes == nullptr) return TT_ERR_INVALID_ARG;
    const tt_status st = check_clip_list(count, n, dtypes);
    if (st != TT_OK) return st;
    *bytes = clip_workspace_bytes({count, nullptr, nullptr, n, dtypes}, sm_count_current());
    return TT_OK;
}

tt_status tt_grad_norm(int32_t count, const void* const* grads, const int64_t* n, const int32_t* dtypes, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream) {
    return clip({count, grads, const_cast<void* const*>(grads), n, dtypes}, false, 0.0f, norm, workspace,
                workspace_bytes, stream);
}

tt_status tt_clip_grad_norm(int32_t count, const void* const* grads, const int64_t* n, const int32_t* dtypes,
                            void* const* out, float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                            void* stream) {
    return clip({count, grads, out != nullptr ? out : const_cast<void* const*>(grads), n, dtypes}, true, max_norm, norm,
                workspace, workspace_bytes, stream);
}

tt_status tt_embedding(const void* table, tt_dtype table_dtype, int64_t rows, int32_t d, const void* ids,
                       int32_t id_bytes, int64_t m, float scale, void* out, tt_dtype out_dtype, void* stream) {
    tt_status st = check_embedding(rows, d, id_bytes, m, scale);
    if (st != TT_OK) return st;
    if (!valid_dtype(table_dtype) || !valid_dtype(out_dtype)) return TT_ERR_INVALID_ARG;
    if (!aligned(table, 16) || !aligned(ids, id_bytes) || !aligned(out, 16)) return TT_ERR_INVALID_ARG;
    if (m == 0) return TT_OK;
    if ((rows > 0 && table == nullptr) || ids == nullptr || out == nullptr) return TT_ERR_INVALID_ARG;
    Buffers b;
    b.in(table, (size_t)rows * d * elem_bytes(table_dtype), "table");
    b.in(ids, (size_t)m * id_bytes, "ids");
    b.out(out, (size_t)m * d * elem_bytes(out_dtype), "out");
    if ((st = b.check()) != TT_OK) return st;
    const cudaError_t e = launch_embedding(table, table_dtype, rows, d, ids, id_bytes, m, scale, out, out_dtype,
                                           static_cast<cudaStream_t>(stream), sm_count_current());
    return e == cudaSuccess ? TT_OK : cuda_fail(e, "embedding lookup");
}

tt_status tt_embedding_grad_workspace(int64_t m, int64_t rows, int32_t d, size_t* bytes) {
    if (bytes == nullptr) return TT_ERR_INVALID_ARG;
    const tt_status st = check_embedding(rows, d, 4, m, 1.0f);
    if (st != TT_OK) return st;
    *bytes = embedding_grad_bytes(m, rows, d);
    return TT_OK;
}

tt_status tt_embedding_grad(const void* ids, int32_t id_bytes, int64_t m, const void* grad, tt_dtype grad_dtype,
                            int64_t rows, int32_t d, float scale, void* grad_table, tt_dtype out_dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
    return embedding_grad({ids, id_bytes, m, rows, grad, grad_dtype, d, scale, grad_table, out_dtype, nullptr, nullptr,
                           workspace},
                          false, workspace_bytes, stream);
}

tt_status tt_embedding_grad_rows(const void* ids, int32_t id_bytes, int64_t m, const void* grad, tt_dtype grad_dtype,
                                 int64_t rows, int32_t d, float scale, void* out_ids, void* out_rows,
                                 tt_dtype out_dtype, int32_t* count, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    return embedding_grad({ids, id_bytes, m, rows, grad, grad_dtype, d, scale, out_rows, out_dtype, out_ids, count,
                           workspace},
                          true, workspace_bytes, stream);
}

static tt_status softmax_grad_sizes(int32_t b, int32_t nc, int32_t d, bool with_ids) {
    if (b < 0 || nc < b || d <= 0) return TT_ERR_INVALID_ARG;
    if (d % 16 != 0 || d < 64 || d > TT_MAX_D) return TT_ERR_UNSUPPORTED;
    if (nc > (with_ids ? 1 << 28 : 1 << 30)) return TT_ERR_UNSUPPORTED;
    return TT_OK;
}

tt_status tt_inbatch_softmax_grad_workspace(int32_t b, int32_t nc, int32_t d, int32_t with_item_ids,
                                            int32_t with_valid, size_t* bytes) {
    if (bytes == nullptr) return TT_ERR_INVALID_ARG;
    const tt_status st = softmax_grad_sizes(b, nc, d, with_item_ids != 0);
    if (st != TT_OK) return st;
    *bytes = softmax_grad_plan(b, nc, d, with_item_ids != 0, with_valid != 0, sm_count_current()).bytes;
    return TT_OK;
}

tt_status tt_inbatch_softmax_grad(const void* users, const void* items, tt_dtype dtype, int32_t b, int32_t nc,
                                  int32_t d, float tau, const float* logq, const int64_t* item_ids,
                                  const uint8_t* valid, const float* lse, const float* loss, const float* grad_loss,
                                  const float* grad_mean, void* grad_users, void* grad_items, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    if (dtype != TT_BF16) return dtype == TT_F32 || dtype == TT_I8 ? TT_ERR_UNSUPPORTED : TT_ERR_INVALID_ARG;
    tt_status st = softmax_grad_sizes(b, nc, d, item_ids != nullptr);
    if (st != TT_OK) return st;
    if (!(tau > 0.0f) || !isfinite(tau)) return TT_ERR_INVALID_ARG;
    if (grad_loss == nullptr && grad_mean == nullptr) return TT_ERR_INVALID_ARG;
    if (b > 0 && (users == nullptr || lse == nullptr || loss == nullptr || grad_users == nullptr)) return TT_ERR_INVALID_ARG;
    if (nc > 0 && (items == nullptr || grad_items == nullptr)) return TT_ERR_INVALID_ARG;
    if (!aligned(users, 16) || !aligned(items, 16) || !aligned(grad_users, 16) || !aligned(grad_items, 16) ||
        !aligned(logq, 4) || !aligned(item_ids, 8) || !aligned(lse, 4) || !aligned(loss, 4) || !aligned(grad_loss, 4) ||
        !aligned(grad_mean, 4))
        return TT_ERR_INVALID_ARG;
    const int sms = sm_count_current();
    const SoftmaxGradPlan pl = softmax_grad_plan(b, nc, d, item_ids != nullptr, valid != nullptr, sms);
    if ((st = check_workspace(workspace, workspace_bytes, pl.bytes)) != TT_OK) return st;
    const size_t u_bytes = (size_t)b * d * 2, v_bytes = (size_t)nc * d * 2;
    Buffers k;
    k.in(users, u_bytes, "users");
    k.in(items, v_bytes, "items");
    k.in(logq, nc * sizeof(float), "logq");
    k.in(item_ids, nc * sizeof(int64_t), "item_ids");
    k.in(valid, nc, "valid");
    k.in(lse, b * sizeof(float), "lse");
    k.in(loss, b * sizeof(float), "loss");
    k.in(grad_loss, b * sizeof(float), "grad_loss");
    k.in(grad_mean, sizeof(float), "grad_mean");
    k.out(grad_users, u_bytes, "grad_users");
    k.out(grad_items, v_bytes, "grad_items");
    k.out(workspace, pl.bytes, "workspace");
    if ((st = k.check()) != TT_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (b == 0) {  // no rows: no sums; the error word says that nothing failed
        TT_CUDA(cudaMemsetAsync(workspace, 0, sizeof(int), s), "error word");
        if (nc > 0) TT_CUDA(cudaMemsetAsync(grad_items, 0, v_bytes, s), "item gradients");
        return TT_OK;
    }
    SoftmaxGrad g;
    memset(&g, 0, sizeof g);
    const uint8_t* ws = static_cast<const uint8_t*>(workspace);
    const void* u_src = valid != nullptr ? ws + pl.off_users_c : users;
    const void* v_src = valid != nullptr ? ws + pl.off_items_c : items;
    if (!bf16_tile_tensor_map(u_src, b, d, d, 128, &g.tm_ux) || !bf16_tile_tensor_map(u_src, b, d, d, pl.tile_cols, &g.tm_uy) ||
        !bf16_tile_tensor_map(v_src, nc, d, d, 128, &g.tm_vx) || !bf16_tile_tensor_map(v_src, nc, d, d, pl.tile_cols, &g.tm_vy))
        return TT_ERR_CUDA;
    g.users = users;
    g.items = items;
    g.b = b;
    g.nc = nc;
    g.d = d;
    g.tau = tau;
    g.logq = logq;
    g.item_ids = item_ids;
    g.valid = valid;
    g.lse = lse;
    g.loss = loss;
    g.grad_loss = grad_loss;
    g.grad_mean = grad_mean;
    g.grad_users = grad_users;
    g.grad_items = grad_items;
    g.workspace = workspace;
    const cudaError_t e = launch_softmax_grad(pl, g, s, sms);
    return e == cudaSuccess ? TT_OK : cuda_fail(e, "in-batch softmax gradient");
}

}  // extern "C"
