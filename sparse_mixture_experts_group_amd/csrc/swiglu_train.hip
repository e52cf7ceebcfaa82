// SwiGLU between the experts' two products, with the 8-bit copy of its inputs for the
// backward pass, and the backward pass out of that copy.
#include "train_kernels.h"
#include "train_rows.cuh"

namespace beam {

__device__ __forceinline__ Item item_at(const SwigluArgs& a, int64_t k) {
    return item_at(k, a.pairs, a.rows, a.row_of_pair, a.pair_of_row);
}

__device__ __forceinline__ float item_weight(const SwigluArgs& a, const Item& t) {
    return a.weights && t.live ? a.weights[t.pair] : 1.0f;
}

static int64_t items(const SwigluArgs& a) { return a.pair_of_row ? a.rows : a.pairs; }

static void write_pairs_down(hipStream_t st, const SwigluArgs& a, float* dweights) {
    if (a.pair_of_row) launch_invert(st, a.pairs, a.rows, a.row_of_pair, a.pair_of_row, dweights);
}

// sigma(g): the hardware exponential and reciprocal, about 2 ulp; results are rounded to
// BF16 or held to FP32 tolerances.
__device__ __forceinline__ float sigmoid_fast(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// ---------------------------------------------------------------------------
// h[r] = w g sigma(g) u, (g, u) the halves of gu[r].  A thread has 8 columns of g and the
// same of u, four lanes a block of the 8-bit copy.  Bound by HBM: 65536 mapped rows of 2560
// BF16 columns with the copy 227 us (6.0 TB/s; a plain copy reaches 6.65).
// ---------------------------------------------------------------------------
template <bool BF16, bool ALIGNED, bool KEEP>
__global__ __launch_bounds__(256) void swiglu_rows(SwigluArgs a, int pieces, const void* __restrict__ gu,
                                                   void* __restrict__ h, uint8_t* __restrict__ keep_q,
                                                   uint8_t* __restrict__ keep_scale) {
    int64_t k;
    int piece;
    piece_of_thread(pieces, k, piece);
    const int c = piece * 8, n = a.I - c;
    const Item it = item_at(a, k);            // one row for the four lanes of a block
    const int64_t r = it.row;
    const bool here = n > 0;
    float g[8] = {}, u[8] = {};
    if (here && r >= 0) {
        const int64_t at = r * 2 * a.I + c;
        widen8<BF16>(load_raw8<BF16, ALIGNED, true>(gu, at, n), g);
        widen8<BF16>(load_raw8<BF16, ALIGNED, true>(gu, at + a.I, n), u);
    }
    if (!it.live) return;
    if constexpr (KEEP) {
        u32x2 qg, qu;
        const int cg = keep8(g, qg), cu = keep8(u, qu);
        if (here) {
            uint8_t* q = keep_q + r * 2 * a.I + c;
            store_codes8<ALIGNED, true>(q, n, qg);
            store_codes8<ALIGNED, true>(q + a.I, n, qu);
            if ((piece & 3) == 0) {
                const int nb = keep_blocks(a.I);
                uint8_t* s = keep_scale + r * 2 * nb + piece / 4;
                s[0] = static_cast<uint8_t>(cg);
                s[nb] = static_cast<uint8_t>(cu);
            }
        }
    }
    if (!here) return;
    const float w = item_weight(a, it);
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = w * (g[j] * sigmoid_fast(g[j]) * u[j]);
    store_raw8<BF16, ALIGNED, true>(h, r * a.I + c, n, narrow8<BF16>(o));
}

template <bool BF16, bool ALIGNED>
static void swiglu_typed(hipStream_t st, const SwigluArgs& a, const void* gu, void* h, uint8_t* keep_q,
                         uint8_t* keep_scale) {
    const int pieces = (a.I + 31) / 32 * 4;
    const unsigned blocks = static_cast<unsigned>((items(a) * pieces + 255) / 256);
    write_pairs_down(st, a, nullptr);
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
// A thread reads its columns before it writes them, so dgu may lie over an FP32 or BF16 gu,
// and h over dh.  Bound by HBM: from the 8-bit copy, 65536 mapped rows of 2560 BF16 columns
// with dw 300 us (5.6 TB/s), 4096 rows of 20480 without 133 us (6.3).
// ---------------------------------------------------------------------------
// One 8-column piece of a row: its values,
template <bool BF16, bool ALIGNED, bool SRC8>
struct SwigluPiece {
    Raw8<BF16> g, u, d;
    u32x2 qg, qu;
    uint8_t sg, su;

    __device__ __forceinline__ void load(const SwigluArgs& a, int64_t r, int c, const void* dh, const void* gu,
                                         const uint8_t* gu_scale) {
        const int n = a.I - c;
        const int64_t at = r * 2 * a.I + c;
        if constexpr (SRC8) {
            const uint8_t* q = static_cast<const uint8_t*>(gu) + at;
            const int nb = keep_blocks(a.I);
            const uint8_t* s = gu_scale + r * 2 * nb + c / kKeepBlock;
            qg = load_codes8<ALIGNED, true>(q, n);
            qu = load_codes8<ALIGNED, true>(q + a.I, n);
            sg = s[0];
            su = s[nb];
        } else {
            g = load_raw8<BF16, ALIGNED, true>(gu, at, n);
            u = load_raw8<BF16, ALIGNED, true>(gu, at + a.I, n);
        }
        d = load_raw8<BF16, ALIGNED, true>(dh, r * a.I + c, n);
    }

    // and its gradients; returns its part of dw.
    __device__ __forceinline__ float run(const SwigluArgs& a, int64_t r, int c, float w, void* dgu, void* h) const {
        const int n = a.I - c;
        const int64_t at = r * 2 * a.I + c;
        float gf[8], uf[8], df[8];
        if constexpr (SRC8) {
            restore8(qg, keep_scale(sg), gf);
            restore8(qu, keep_scale(su), uf);
        } else {
            widen8<BF16>(g, gf);
            widen8<BF16>(u, uf);
        }
        widen8<BF16>(d, df);
        float dg[8], du[8], o[8], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = sigmoid_fast(gf[j]);
            const float act = gf[j] * s, v = act * uf[j];
            sum = fmaf(df[j], v, sum);
            o[j] = w * v;
            const float e = w * df[j];
            du[j] = e * act;
            dg[j] = e * uf[j] * (s * fmaf(gf[j], 1.0f - s, 1.0f));
        }
        store_raw8<BF16, ALIGNED, true>(dgu, at, n, narrow8<BF16>(dg));
        store_raw8<BF16, ALIGNED, true>(dgu, at + a.I, n, narrow8<BF16>(du));
        if (h) store_raw8<BF16, ALIGNED, true>(h, r * a.I + c, n, narrow8<BF16>(o));
        return sum;
    }
};

// Without the weights' gradient: a thread a piece, rows packed back to back.
template <bool BF16, bool ALIGNED, bool SRC8>
__global__ __launch_bounds__(256) void swiglu_backward_flat(SwigluArgs a, int pieces, const void* dh, const void* gu,
                                                            const uint8_t* __restrict__ gu_scale, void* dgu, void* h) {
    int64_t k;
    int piece;
    piece_of_thread(pieces, k, piece);
    const Item it = item_at(a, k);
    if (it.row < 0) return;
    SwigluPiece<BF16, ALIGNED, SRC8> v;
    v.load(a, it.row, piece * 8, dh, gu, gu_scale);
    if (it.live) v.run(a, it.row, piece * 8, item_weight(a, it), dgu, h);
}

// With it: a group of threads a row (row_group).
template <bool BF16, bool ALIGNED, bool SRC8>
__global__ __launch_bounds__(1024) void swiglu_backward(SwigluArgs a, int group, const void* dh, const void* gu,
                                                        const uint8_t* __restrict__ gu_scale, void* dgu, void* h,
                                                        float* __restrict__ dweights) {
    __shared__ float s_sum[16];
    const int lane = group <= 64 ? threadIdx.x & (group - 1) : threadIdx.x;
    const int64_t k = group <= 64 ? static_cast<int64_t>(blockIdx.x) * (256 / group) + threadIdx.x / group : blockIdx.x;
    const Item it = item_at(a, k);
    float sum = 0.0f;
    if (it.row >= 0) {
        for (int c = lane * 8; c < a.I; c += group * 8) {
            SwigluPiece<BF16, ALIGNED, SRC8> v;
            v.load(a, it.row, c, dh, gu, gu_scale);
            if (it.live) sum += v.run(a, it.row, c, item_weight(a, it), dgu, h);
        }
    }
    sum = group_sum(sum, group, s_sum);
    // in the order of pairs a dropped one's 0 is written here
    if (lane == 0 && (a.pair_of_row ? it.live : k < a.pairs)) dweights[it.pair] = sum;
}

template <bool BF16, bool ALIGNED, bool SRC8>
static void swiglu_backward_typed(hipStream_t st, const SwigluArgs& a, const void* dh, const void* gu,
                                  const uint8_t* gu_scale, void* dgu, void* h, float* dweights) {
    write_pairs_down(st, a, dweights);
    if (dweights) {
        // 65536 rows of 2560 columns: 299 us with a piece a thread (320 threads), 349 with a
        // wave a row; rows in order keep even large blocks' addresses close together
        const int group = row_group(a.I, 1024);
        swiglu_backward<BF16, ALIGNED, SRC8><<<group_blocks(items(a), group), group_threads(group), 0, st>>>(
            a, group, dh, gu, gu_scale, dgu, h, dweights);
    } else {
        const int pieces = (a.I + 7) / 8;
        const unsigned blocks = static_cast<unsigned>((items(a) * pieces + 255) / 256);
        swiglu_backward_flat<BF16, ALIGNED, SRC8><<<blocks, 256, 0, st>>>(a, pieces, dh, gu, gu_scale, dgu, h);
    }
}

template <bool BF16, bool ALIGNED>
static void swiglu_backward_from(hipStream_t st, const SwigluArgs& a, const void* dh, const void* gu,
                                 const uint8_t* gu_scale, void* dgu, void* h, float* dweights) {
    if (gu_scale) swiglu_backward_typed<BF16, ALIGNED, true>(st, a, dh, gu, gu_scale, dgu, h, dweights);
    else swiglu_backward_typed<BF16, ALIGNED, false>(st, a, dh, gu, nullptr, dgu, h, dweights);
}

void launch_swiglu_backward(hipStream_t st, const SwigluArgs& a, const void* dh, const void* gu,
                            const uint8_t* gu_scale, void* dgu, void* h, float* dweights) {
    if (a.pairs == 0) return;
    const bool al = a.I % 8 == 0;
    if (a.bf16 && al) swiglu_backward_from<true, true>(st, a, dh, gu, gu_scale, dgu, h, dweights);
    else if (a.bf16) swiglu_backward_from<true, false>(st, a, dh, gu, gu_scale, dgu, h, dweights);
    else if (al) swiglu_backward_from<false, true>(st, a, dh, gu, gu_scale, dgu, h, dweights);
    else swiglu_backward_from<false, false>(st, a, dh, gu, gu_scale, dgu, h, dweights);
}

}  // namespace beam
