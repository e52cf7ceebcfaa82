// SwiGLU between the experts' two products, with the 8-bit copy of its inputs for the
// backward pass, and the backward pass out of that copy.
#include "train_kernels.h"
#include "train_rows.cuh"

namespace beam {

__device__ __forceinline__ int64_t row_of(const SwigluArgs& a, int64_t p) {
    const int64_t r = a.row_of_pair ? a.row_of_pair[p] : p;
    return r >= 0 && r < a.rows ? r : -1;
}

// sigma(g): the hardware exponential and reciprocal, about 2 ulp; results are rounded to
// BF16 or held to FP32 tolerances.
__device__ __forceinline__ float sigmoid_fast(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// ---------------------------------------------------------------------------
// h[r] = w g sigma(g) u, (g, u) the halves of gu[r].  A thread has 8 columns of g and the
// same of u.
// ---------------------------------------------------------------------------
template <bool BF16, bool ALIGNED, bool KEEP>
__global__ __launch_bounds__(256) void swiglu_rows(SwigluArgs a, int pieces, const void* __restrict__ gu,
                                                   void* __restrict__ h, uint8_t* __restrict__ keep_q,
                                                   uint8_t* __restrict__ keep_scale) {
    int64_t p;
    int piece;
    piece_of_thread(pieces, p, piece);
    const int c = piece * 8, n = a.I - c;
    const int64_t r = p < a.pairs ? row_of(a, p) : -1;      // one row for the four lanes of a block
    if (r < 0) return;
    const bool here = n > 0;
    float g[8] = {}, u[8] = {};
    if (here) {
        const int64_t at = r * 2 * a.I + c;
        widen8<BF16>(load_raw8<BF16, ALIGNED>(gu, at, n), g);
        widen8<BF16>(load_raw8<BF16, ALIGNED>(gu, at + a.I, n), u);
    }
    if constexpr (KEEP) {
        u32x2 qg, qu;
        const int cg = keep8(g, qg), cu = keep8(u, qu);
        if (here) {
            uint8_t* q = keep_q + r * 2 * a.I + c;
            store_codes8<ALIGNED>(q, n, qg);
            store_codes8<ALIGNED>(q + a.I, n, qu);
            if ((piece & 3) == 0) {
                const int nb = keep_blocks(a.I);
                uint8_t* s = keep_scale + r * 2 * nb + piece / 4;
                s[0] = static_cast<uint8_t>(cg);
                s[nb] = static_cast<uint8_t>(cu);
            }
        }
    }
    if (!here) return;
    const float w = a.weights ? a.weights[p] : 1.0f;
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = w * (g[j] * sigmoid_fast(g[j]) * u[j]);
    store_raw8<BF16, ALIGNED>(h, r * a.I + c, n, narrow8<BF16>(o));
}

template <bool BF16, bool ALIGNED>
static void swiglu_typed(hipStream_t st, const SwigluArgs& a, const void* gu, void* h, uint8_t* keep_q,
                         uint8_t* keep_scale) {
    const int pieces = (a.I + 31) / 32 * 4;
    const unsigned blocks = static_cast<unsigned>((a.pairs * pieces + 255) / 256);
    if (keep_q) swiglu_rows<BF16, ALIGNED, true><<<blocks, 256, 0, st>>>(a, pieces, gu, h, keep_q, keep_scale);
    else swiglu_rows<BF16, ALIGNED, false><<<blocks, 256, 0, st>>>(a, pieces, gu, h, nullptr, nullptr);
}

void launch_swiglu(hipStream_t st, const SwigluArgs& a, const void* gu, void* h, uint8_t* keep_q, uint8_t* keep_scale) {
    if (a.pairs == 0) return;
    const bool al = a.I % 8 == 0;
    if (a.bf16 && al) swiglu_typed<true, true>(st, a, gu, h, keep_q, keep_scale);
    else if (a.bf16) swiglu_typed<true, false>(st, a, gu, h, keep_q, keep_scale);
    else if (al) swiglu_typed<false, true>(st, a, gu, h, keep_q, keep_scale);
    else swiglu_typed<false, false>(st, a, gu, h, keep_q, keep_scale);
}

// ---------------------------------------------------------------------------
// backward: with s = sigma(g), a = g s:
//   dg = w dh u s (1 + g (1 - s)),  du = w dh a,  h = w a u (again, for the down weights'
//   gradient),  dw = sum over the row of dh a u.
// `group` threads share a row (as in the gradient of combine).  A thread reads its
// columns before it writes them, so dgu may lie over an FP32 or BF16 gu, and h over dh.
// ---------------------------------------------------------------------------
template <bool BF16, bool ALIGNED, bool SRC8>
__global__ __launch_bounds__(256) void swiglu_backward(SwigluArgs a, int group, const void* dh, const void* gu,
                                                       const uint8_t* __restrict__ gu_scale, void* dgu, void* h,
                                                       float* __restrict__ dweights) {
    __shared__ float s_sum[4];
    const int lane = threadIdx.x & (group - 1);
    const int64_t p = static_cast<int64_t>(blockIdx.x) * (256 / group) + threadIdx.x / group;
    const int64_t r = p < a.pairs ? row_of(a, p) : -1;
    float sum = 0.0f;
    if (r >= 0) {
        const float w = a.weights ? a.weights[p] : 1.0f;
        for (int c = lane * 8; c < a.I; c += group * 8) {
            const int n = a.I - c;
            const int64_t at = r * 2 * a.I + c;
            float g[8], u[8], d[8];
            if constexpr (SRC8) {
                const uint8_t* q = static_cast<const uint8_t*>(gu) + at;
                const int nb = keep_blocks(a.I);
                const uint8_t* s = gu_scale + r * 2 * nb + c / kKeepBlock;
                restore8(load_codes8<ALIGNED>(q, n), keep_scale(s[0]), g);
                restore8(load_codes8<ALIGNED>(q + a.I, n), keep_scale(s[nb]), u);
            } else {
                widen8<BF16>(load_raw8<BF16, ALIGNED>(gu, at, n), g);
                widen8<BF16>(load_raw8<BF16, ALIGNED>(gu, at + a.I, n), u);
            }
            widen8<BF16>(load_raw8<BF16, ALIGNED>(dh, r * a.I + c, n), d);
            float dg[8], du[8], o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float s = sigmoid_fast(g[j]);
                const float act = g[j] * s, v = act * u[j];
                sum = fmaf(d[j], v, sum);
                o[j] = w * v;
                const float e = w * d[j];
                du[j] = e * act;
                dg[j] = e * u[j] * (s * fmaf(g[j], 1.0f - s, 1.0f));
            }
            store_raw8<BF16, ALIGNED>(dgu, at, n, narrow8<BF16>(dg));
            store_raw8<BF16, ALIGNED>(dgu, at + a.I, n, narrow8<BF16>(du));
            if (h) store_raw8<BF16, ALIGNED>(h, r * a.I + c, n, narrow8<BF16>(o));
        }
    }
    if (!dweights) return;
    const int inside = group < 64 ? group : 64;
    for (int o = inside >> 1; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    if (group > 64) {
        if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
        __syncthreads();
        sum = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
    }
    if (lane == 0 && p < a.pairs) dweights[p] = sum;         // 0 for a dropped pair
}

template <bool BF16, bool ALIGNED>
static void swiglu_backward_typed(hipStream_t st, const SwigluArgs& a, int group, const void* dh, const void* gu,
                                  const uint8_t* gu_scale, void* dgu, void* h, float* dweights) {
    const unsigned blocks = static_cast<unsigned>((a.pairs + 256 / group - 1) / (256 / group));
    if (gu_scale)
        swiglu_backward<BF16, ALIGNED, true><<<blocks, 256, 0, st>>>(a, group, dh, gu, gu_scale, dgu, h, dweights);
    else
        swiglu_backward<BF16, ALIGNED, false><<<blocks, 256, 0, st>>>(a, group, dh, gu, nullptr, dgu, h, dweights);
}

void launch_swiglu_backward(hipStream_t st, const SwigluArgs& a, const void* dh, const void* gu,
                            const uint8_t* gu_scale, void* dgu, void* h, float* dweights) {
    if (a.pairs == 0) return;
    const int group = row_group(a.pairs, a.I);
    const bool al = a.I % 8 == 0;
    if (a.bf16 && al) swiglu_backward_typed<true, true>(st, a, group, dh, gu, gu_scale, dgu, h, dweights);
    else if (a.bf16) swiglu_backward_typed<true, false>(st, a, group, dh, gu, gu_scale, dgu, h, dweights);
    else if (al) swiglu_backward_typed<false, true>(st, a, group, dh, gu, gu_scale, dgu, h, dweights);
    else swiglu_backward_typed<false, false>(st, a, group, dh, gu, gu_scale, dgu, h, dweights);
}

}  // namespace beam
