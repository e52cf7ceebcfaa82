// C ABI of the training operators: validation and launches.  The declarations and the
// contract of every entry point are in beam_moe.h.
#include <math.h>

#include "beam_moe.h"
#include "kernels.h"
#include "train_kernels.h"
#include "train_rows.cuh"

using namespace beam;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A pointer that must be there, or may be null, and is 16-byte aligned.
bool given(const void* p) { return p && aligned16(p); }
bool optional(const void* p) { return !p || aligned16(p); }

// Elements of one array: their offsets in bytes stay far from 64 bits.
constexpr int64_t kMaxElements = int64_t{1} << 40;
// Threads of one launch: a grid's are counted in 32 bits, and fill whole blocks.
constexpr int64_t kMaxThreads = (int64_t{1} << 32) - 1024;
// Columns of a row: kernels count them in 32 bits, with a block's stride beyond the end.
constexpr int64_t kMaxWidth = int64_t{1} << 28;

// Tokens, picks and (width >= 0) a row width that an operator takes.
int check_pairs(const beam_moe_config* c, int64_t T, int64_t width) {
    if (!c || T < 0) return BEAM_ERR_INVALID_ARG;
    if (c->topk < 1 || c->topk > kMaxTopK) return BEAM_ERR_INVALID_ARG;
    if (T > INT32_MAX / 2 / c->topk) return BEAM_ERR_INVALID_ARG;
    if (width < 1 || width > kMaxWidth) return BEAM_ERR_INVALID_ARG;
    if (T > 0 && width > kMaxElements / T / c->topk) return BEAM_ERR_INVALID_ARG;
    return BEAM_OK;
}

int check_act(const beam_moe_config* c) {
    if (c->act_dtype < BEAM_DTYPE_F32 || c->act_dtype > BEAM_DTYPE_FP8_E4M3) return BEAM_ERR_INVALID_ARG;
    return c->act_dtype == BEAM_DTYPE_FP8_E4M3 ? BEAM_ERR_UNSUPPORTED : BEAM_OK;
}

int check_rows_call(const beam_moe_config* c, int64_t T, int64_t rows) {
    int s = check_pairs(c, T, c ? c->hidden : 0);
    if (s != BEAM_OK) return s;
    if (rows < 0 || rows > INT32_MAX || rows > kMaxElements / c->hidden) return BEAM_ERR_INVALID_ARG;
    if (T > kMaxThreads / row_threads(c->hidden)) return BEAM_ERR_INVALID_ARG;
    return check_act(c);
}

RowArgs row_args(const beam_moe_config* c, int64_t T, int64_t rows, const int32_t* row_of_pair, const float* weights) {
    return RowArgs{T, rows, c->hidden, c->topk, c->act_dtype == BEAM_DTYPE_BF16, row_of_pair, weights};
}

int launched() { return hipGetLastError() == hipSuccess ? BEAM_OK : BEAM_ERR_HIP; }

size_t sort_ws(int64_t pairs) { return sizeof(int32_t) * static_cast<size_t>(sort_blocks(pairs)) * kMaxExperts; }

int check_experts(const beam_moe_config* c) {
    return c->n_experts >= 1 && c->n_experts <= kMaxExperts ? BEAM_OK : BEAM_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

size_t beam_moe_sort_workspace_size(const beam_moe_config* cfg, int64_t T) {
    if (check_pairs(cfg, T, 1) != BEAM_OK || check_experts(cfg) != BEAM_OK) return 0;
    return sort_ws(T * cfg->topk);
}

int beam_moe_sort(const beam_moe_config* cfg, int64_t T, const int32_t* ids, int32_t* expert_off,
                  int32_t* row_of_pair, int32_t* pair_of_row, void* ws, size_t ws_bytes, void* stream) {
    int s = check_pairs(cfg, T, 1);
    if (s != BEAM_OK) return s;
    if ((s = check_experts(cfg)) != BEAM_OK) return s;
    if (!given(expert_off)) return BEAM_ERR_INVALID_ARG;
    if (T > 0 && (!given(ids) || !given(row_of_pair) || !given(pair_of_row))) return BEAM_ERR_INVALID_ARG;
    const int64_t pairs = T * cfg->topk;
    const size_t need = sort_ws(pairs);
    if (need > 0) {
        if (!ws || ws_bytes < need) return BEAM_ERR_WORKSPACE;
        if (!aligned16(ws)) return BEAM_ERR_INVALID_ARG;
    }
    (void)hipGetLastError();
    launch_sort_pairs(static_cast<hipStream_t>(stream), pairs, cfg->n_experts, ids, expert_off, row_of_pair,
                      pair_of_row, static_cast<int32_t*>(ws));
    return launched();
}

int beam_moe_dispatch(const beam_moe_config* cfg, int64_t T, const void* x, const uint8_t* x_scale,
                      const int32_t* row_of_pair, int64_t rows, void* xs, uint8_t* keep_q, uint8_t* keep_scale,
                      void* stream) {
    int s = check_rows_call(cfg, T, rows);
    if (s != BEAM_OK) return s;
    if (T == 0) return BEAM_OK;
    if (!row_of_pair && cfg->topk != 1) return BEAM_ERR_INVALID_ARG;
    if ((keep_q != nullptr) != (keep_scale != nullptr) || (keep_q && x_scale)) return BEAM_ERR_INVALID_ARG;
    if (!given(x) || !optional(x_scale) || !optional(row_of_pair)) return BEAM_ERR_INVALID_ARG;
    if (!optional(xs) || !optional(keep_q) || !optional(keep_scale)) return BEAM_ERR_INVALID_ARG;
    if (rows == 0) xs = nullptr;              // no row can be written
    if (!xs && !keep_q) return rows == 0 ? BEAM_OK : BEAM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    launch_dispatch(static_cast<hipStream_t>(stream), row_args(cfg, T, rows, row_of_pair, nullptr), x, x_scale, xs,
                    keep_q, keep_scale);
    return launched();
}

int beam_moe_dispatch_backward(const beam_moe_config* cfg, int64_t T, const void* dxs, const int32_t* row_of_pair,
                               int64_t rows, void* dx, void* stream) {
    int s = check_rows_call(cfg, T, rows);
    if (s != BEAM_OK) return s;
    if (T == 0) return BEAM_OK;
    if (!given(row_of_pair) || !given(dx) || (rows > 0 ? !given(dxs) : !optional(dxs))) return BEAM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    launch_combine_rows(static_cast<hipStream_t>(stream), row_args(cfg, T, rows, row_of_pair, nullptr), dxs, dx);
    return launched();
}

int beam_moe_combine(const beam_moe_config* cfg, int64_t T, const void* expert_out, const int32_t* row_of_pair,
                     int64_t rows, const float* weights, void* y, void* stream) {
    int s = check_rows_call(cfg, T, rows);
    if (s != BEAM_OK) return s;
    if (T == 0) return BEAM_OK;
    if (!given(row_of_pair) || !given(y) || !given(weights)) return BEAM_ERR_INVALID_ARG;
    if (rows > 0 ? !given(expert_out) : !optional(expert_out)) return BEAM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    launch_combine_rows(static_cast<hipStream_t>(stream), row_args(cfg, T, rows, row_of_pair, weights), expert_out, y);
    return launched();
}

int beam_moe_combine_backward(const beam_moe_config* cfg, int64_t T, const void* dy, const void* expert_out,
                              const int32_t* row_of_pair, int64_t rows, const float* weights, void* dexpert_out,
                              float* dweights, void* stream) {
    int s = check_rows_call(cfg, T, rows);
    if (s != BEAM_OK) return s;
    if (T == 0) return BEAM_OK;
    if (!given(dy) || !given(row_of_pair) || !given(weights)) return BEAM_ERR_INVALID_ARG;
    if (rows > 0 ? !given(dexpert_out) : !optional(dexpert_out)) return BEAM_ERR_INVALID_ARG;
    if (!optional(expert_out) || !optional(dweights)) return BEAM_ERR_INVALID_ARG;
    if ((expert_out != nullptr) != (dweights != nullptr)) return BEAM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    launch_combine_backward(static_cast<hipStream_t>(stream), row_args(cfg, T, rows, row_of_pair, weights), dy,
                            expert_out, dexpert_out, dweights);
    return launched();
}

static int check_swiglu(const beam_moe_config* cfg, int64_t T, const int32_t* row_of_pair, int64_t rows) {
    int s = check_pairs(cfg, T, cfg ? cfg->inter : 0);
    if (s != BEAM_OK) return s;
    if (rows < 0 || rows > INT32_MAX || rows > kMaxElements / cfg->inter) return BEAM_ERR_INVALID_ARG;
    const int64_t pairs = T * cfg->topk, items = rows_in_order(pairs, rows, cfg->inter) && rows > pairs ? rows : pairs;
    if (items > kMaxThreads / row_threads(cfg->inter)) return BEAM_ERR_INVALID_ARG;
    if (T > 0 && !row_of_pair && cfg->topk != 1) return BEAM_ERR_INVALID_ARG;
    return check_act(cfg);
}

static SwigluArgs swiglu_args(const beam_moe_config* c, int64_t T, int64_t rows, const int32_t* row_of_pair,
                              const float* weights, void* ws) {
    return SwigluArgs{T * c->topk, rows,    c->inter, c->act_dtype == BEAM_DTYPE_BF16,
                      row_of_pair, weights, static_cast<int32_t*>(ws)};
}

// Workspace of a SwiGLU call that takes rows in order.
static size_t swiglu_ws(const beam_moe_config* c, int64_t T, int64_t rows) {
    return rows_in_order(T * c->topk, rows, c->inter) ? sizeof(int32_t) * static_cast<size_t>(rows) : 0;
}

size_t beam_moe_swiglu_workspace_size(const beam_moe_config* cfg, int64_t T, int64_t rows) {
    if (check_pairs(cfg, T, cfg ? cfg->inter : 0) != BEAM_OK || rows < 0 || rows > INT32_MAX) return 0;
    return swiglu_ws(cfg, T, rows);
}

// The call's workspace in *ws (null where it needs none), or an error.
static int check_swiglu_ws(const beam_moe_config* cfg, int64_t T, int64_t rows, const int32_t* row_of_pair, void** ws,
                           size_t ws_bytes) {
    const size_t need = row_of_pair ? swiglu_ws(cfg, T, rows) : 0;
    if (need == 0) {
        *ws = nullptr;
        return BEAM_OK;
    }
    if (!*ws || ws_bytes < need) return BEAM_ERR_WORKSPACE;
    return aligned16(*ws) ? BEAM_OK : BEAM_ERR_INVALID_ARG;
}

int beam_moe_swiglu(const beam_moe_config* cfg, int64_t T, const void* gu, const int32_t* row_of_pair, int64_t rows,
                    const float* weights, void* h, uint8_t* keep_q, uint8_t* keep_scale, void* ws, size_t ws_bytes,
                    void* stream) {
    int s = check_swiglu(cfg, T, row_of_pair, rows);
    if (s != BEAM_OK) return s;
    if ((keep_q != nullptr) != (keep_scale != nullptr)) return BEAM_ERR_INVALID_ARG;
    if (T == 0 || rows == 0) return BEAM_OK;
    if (!given(gu) || !given(h)) return BEAM_ERR_INVALID_ARG;
    if (!optional(row_of_pair) || !optional(weights) || !optional(keep_q) || !optional(keep_scale))
        return BEAM_ERR_INVALID_ARG;
    if ((s = check_swiglu_ws(cfg, T, rows, row_of_pair, &ws, ws_bytes)) != BEAM_OK) return s;
    (void)hipGetLastError();
    launch_swiglu(static_cast<hipStream_t>(stream), swiglu_args(cfg, T, rows, row_of_pair, weights, ws), gu, h, keep_q,
                  keep_scale);
    return launched();
}

int beam_moe_swiglu_backward(const beam_moe_config* cfg, int64_t T, const void* dh, const void* gu,
                             const uint8_t* gu_scale, const int32_t* row_of_pair, int64_t rows, const float* weights,
                             void* dgu, void* h, float* dweights, void* ws, size_t ws_bytes, void* stream) {
    int s = check_swiglu(cfg, T, row_of_pair, rows);
    if (s != BEAM_OK) return s;
    if (dweights && !weights) return BEAM_ERR_INVALID_ARG;
    if (T == 0) return BEAM_OK;
    if (rows > 0 && (!given(dh) || !given(gu) || !given(dgu))) return BEAM_ERR_INVALID_ARG;
    if (!optional(gu_scale) || !optional(row_of_pair) || !optional(weights) || !optional(h) || !optional(dweights))
        return BEAM_ERR_INVALID_ARG;
    if ((s = check_swiglu_ws(cfg, T, rows, row_of_pair, &ws, ws_bytes)) != BEAM_OK) return s;
    (void)hipGetLastError();
    launch_swiglu_backward(static_cast<hipStream_t>(stream), swiglu_args(cfg, T, rows, row_of_pair, weights, ws), dh, gu,
                           gu_scale, dgu, h, dweights);
    return launched();
}

static int check_route_backward(const beam_moe_config* cfg, int64_t T) {
    int s = check_pairs(cfg, T, cfg ? cfg->hidden : 0);
    if (s != BEAM_OK) return s;
    if ((s = check_experts(cfg)) != BEAM_OK) return s;
    if (!isfinite(cfg->routed_scale)) return BEAM_ERR_INVALID_ARG;
    if ((s = check_act(cfg)) != BEAM_OK) return s;
    return cfg->hidden > (1 << 20) ? BEAM_ERR_UNSUPPORTED : BEAM_OK;
}

size_t beam_moe_route_backward_workspace_size(const beam_moe_config* cfg, int64_t T) {
    if (check_route_backward(cfg, T) != BEAM_OK) return 0;
    return route_backward_plan(T, cfg->hidden, cfg->n_experts, cfg->topk).total;
}

int beam_moe_route_backward(const beam_moe_config* cfg, int64_t T, const void* x, const float* w_router,
                            const float* logits, const int32_t* ids, const float* dweights, const void* dx_add,
                            void* dx, float* dw_router, float* dlogit_bias, void* ws, size_t ws_bytes, void* stream) {
    int s = check_route_backward(cfg, T);
    if (s != BEAM_OK) return s;
    if (!given(dw_router) || !optional(dlogit_bias)) return BEAM_ERR_INVALID_ARG;
    if (T > 0) {
        if (!given(x) || !given(w_router) || !given(logits) || !given(ids) || !given(dweights))
            return BEAM_ERR_INVALID_ARG;
        if (!optional(dx_add) || !optional(dx) || (dx_add && !dx)) return BEAM_ERR_INVALID_ARG;
    }
    const RouteBackwardPlan plan = route_backward_plan(T, cfg->hidden, cfg->n_experts, cfg->topk);
    if (plan.total > 0) {
        if (!ws || ws_bytes < plan.total) return BEAM_ERR_WORKSPACE;
        if (!aligned16(ws)) return BEAM_ERR_INVALID_ARG;
    }
    (void)hipGetLastError();
    launch_route_backward(static_cast<hipStream_t>(stream),
                          RouteBackwardArgs{T, cfg->hidden, cfg->n_experts, cfg->topk, cfg->routed_scale,
                                            cfg->act_dtype == BEAM_DTYPE_BF16},
                          plan, x, w_router, logits, ids, dweights, dx_add, dx, dw_router, dlogit_bias, ws);
    return launched();
}

}  // extern "C"
