// Launchers of the training operators (dispatch, combine, SwiGLU with an 8-bit copy,
// router gradient).  Arguments have been checked by train_api.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace beam {

// ---- sort (dispatch.hip) --------------------------------------------------
// A batch of at most kSortSingle pairs is sorted by one launch of one block, a larger one by
// at most kSortBlocks blocks (count, scatter) with a workspace of their counts.  256 experts:
// one block takes 2.7 us for 128 pairs, 6.8 for 4096, 11.0 for 8192; two launches 7.7, 8.1
// and, for 262144, 13.0.
constexpr int kSortSingle = 4096;
constexpr int kSortBlocks = 256;
inline int64_t sort_chunk(int64_t pairs) {
    const int64_t c = (pairs + kSortBlocks - 1) / kSortBlocks;
    return c <= 1024 ? 1024 : (c + 255) / 256 * 256;
}
inline int64_t sort_blocks(int64_t pairs) {
    return pairs <= kSortSingle ? 0 : (pairs + sort_chunk(pairs) - 1) / sort_chunk(pairs);
}

// counts: [sort_blocks, 256] int32 of workspace (unused for one block).
void launch_sort_pairs(hipStream_t st, int64_t pairs, int E, const int32_t* ids, int32_t* expert_off,
                       int32_t* row_of_pair, int32_t* pair_of_row, int32_t* counts);

// ---- rows (dispatch.hip) --------------------------------------------------
// Values of h from which the SwiGLU operators take rows in order; they need a workspace of
// an int32 a row then.  Forward and backward from the 8-bit copy, in the order of pairs
// against that of rows: 16384 pairs of 512 columns 14.9 and 18.8 us against 16.8 and 20.2,
// 32768 of 512 27.9 and 34.9 against 27.8 and 33.3, 8192 of 2560 34.8 and 44.1 against 33.3
// and 42.3, 65536 of 2560 266 and 337 against 233 and 303.
constexpr int64_t kRowOrderValues = int64_t{1} << 24;
// Rows in order are read whether they have a pair or not: not where more than a quarter of
// a buffer is room to spare.  65536 pairs of 2560 columns, forward and backward, pairs
// against rows: 1.15 rows a pair 261 and 331 us against 244 and 322, 1.25 257 and 326
// against 256 and 332, 1.5 254 and 328 against 278 and 354, 2 256 and 325 against 330 and
// 404.  With half as many rows as pairs (the rest on other devices) 148 and 217 against 132
// and 173.
inline bool rows_in_order(int64_t pairs, int64_t rows, int64_t cols) {
    return pairs * cols >= kRowOrderValues && rows * 4 <= pairs * 5;
}

// pair_of_row [rows] from row_of_pair [pairs]; a dropped pair's dweights (if given) are zeros.
void launch_invert(hipStream_t st, int64_t pairs, int64_t rows, const int32_t* row_of_pair, int32_t* pair_of_row,
                   float* dweights);

struct RowArgs {
    int64_t T;                   // tokens
    int64_t rows;                // rows of the sorted buffers
    int H, K;
    bool bf16;
    const int32_t* row_of_pair;  // [T, K], or null: K = 1 and row = token
    const float* weights;        // [T, K] or null (ones)
};

// xs[row] = x[t] (x_scale: x holds E4M3 codes); keep_q / keep_scale: the 8-bit copy of x.
void launch_dispatch(hipStream_t st, const RowArgs& a, const void* x, const uint8_t* x_scale, void* xs,
                     uint8_t* keep_q, uint8_t* keep_scale);
// y[t] = sum_i w_i in[row_i]
void launch_combine_rows(hipStream_t st, const RowArgs& a, const void* in, void* y);
// deo[row_i] = w_i dy[t], dweights[t, i] = <dy[t], eo[row_i]> (eo null: deo only)
void launch_combine_backward(hipStream_t st, const RowArgs& a, const void* dy, const void* eo, void* deo,
                             float* dweights);

// ---- SwiGLU (swiglu_train.hip) ---------------------------------------------
struct SwigluArgs {
    int64_t pairs;               // pairs (rows of the dense MLP)
    int64_t rows;                // rows of the buffers
    int I;
    bool bf16;
    const int32_t* row_of_pair;  // [pairs] or null: row = pair
    const float* weights;        // [pairs] or null (ones)
    int32_t* pair_of_row;        // [rows] of workspace: rows are taken in order; or null: pairs are
};

void launch_swiglu(hipStream_t st, const SwigluArgs& a, const void* gu, void* h, uint8_t* keep_q, uint8_t* keep_scale);
// gu_scale: gu holds E4M3 codes.  h and dweights may be null.
void launch_swiglu_backward(hipStream_t st, const SwigluArgs& a, const void* dh, const void* gu,
                            const uint8_t* gu_scale, void* dgu, void* h, float* dweights);

// ---- router gradient (route_backward.hip) ----------------------------------
struct RouteBackwardArgs {
    int64_t T;
    int H, E, K;
    float alpha;
    bool bf16;                   // x, dx_add, dx
};

struct RouteBackwardPlan {
    int splits;                  // token ranges whose partial dW_r are added up
    size_t dz, expert, split, live, part, total;   // workspace offsets and size
};
RouteBackwardPlan route_backward_plan(int64_t T, int H, int E, int K);
void launch_route_backward(hipStream_t st, const RouteBackwardArgs& a, const RouteBackwardPlan& plan, const void* x,
                           const float* w_router, const float* logits, const int32_t* ids, const float* dweights,
                           const void* dx_add, void* dx, float* dw_router, float* dlogit_bias, void* ws);

}  // namespace beam
