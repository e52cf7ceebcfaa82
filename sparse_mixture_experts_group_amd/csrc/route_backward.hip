// Gradient of the router: from the combine weights' gradients through the normalised
// sigmoid scores to the activations, the router's weights and the logits' bias.
#include "common.cuh"
#include "kernels.h"
#include "train_kernels.h"
#include "train_rows.cuh"

namespace beam {

namespace {

constexpr int kColTile = 128;      // hidden columns of one block
constexpr int kDxStride = kColTile + 2;
constexpr int kDwStride = kColTile + 1;
constexpr int kCUs = 256;

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

RouteBackwardPlan route_backward_plan(int64_t T, int H, int E, int K) {
    RouteBackwardPlan p;
    const int64_t tiles = (static_cast<int64_t>(H) + 1 + kColTile - 1) / kColTile;   // a column for the bias
    int64_t s = kCUs / tiles;
    if (s > (T + 63) / 64) s = (T + 63) / 64;
    if (s < 1) s = 1;
    if (T == 0) s = 0;
    p.splits = static_cast<int>(s);
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off += align256(bytes); return o; };
    p.dz = take(sizeof(float) * T * K);
    p.expert = take(sizeof(int32_t) * T * K);
    p.part = take(sizeof(float) * p.splits * (static_cast<size_t>(H) + 1) * E);
    p.total = off;
    return p;
}

// ---------------------------------------------------------------------------
// dz: with s_i = sigma(z_i), p_i = s_i / sum_j s_j and w_i = alpha p_i,
//   dz_i = alpha p_i (1 - s_i) sum_j p_j (g_i - g_j),
// g the weights' gradients.  The sum over differences loses nothing when the g are nearly
// equal, and 1 - s_i = sigma(-z_i) nothing when s_i is near one.  A lane a pick, `group`
// lanes (a power of two, at least K) a token.  An id outside [0, E) is no pick.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void route_dz(RouteBackwardArgs a, int group, const float* __restrict__ logits,
                                                const int32_t* __restrict__ ids, const float* __restrict__ dweights,
                                                float* __restrict__ dz, int32_t* __restrict__ expert) {
    const int64_t g0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t t = g0 / group;
    const int i = static_cast<int>(threadIdx.x) & (group - 1);
    const int base = (threadIdx.x & 63) & ~(group - 1);
    const bool here = t < a.T && i < a.K;
    const int e = here ? ids[t * a.K + i] : -1;
    const bool live = e >= 0 && e < a.E;
    const float z = live ? logits[t * a.E + e] : 0.0f;
    const float s = live ? router_sigmoid(z) : 0.0f;
    const float g = live ? dweights[t * a.K + i] : 0.0f;
    float d = 0.0f;
    for (int k = 0; k < a.K; ++k) d += __shfl(s, base + k, kWave);
    const float p = live ? s / d : 0.0f;
    float sum = 0.0f;
    for (int k = 0; k < a.K; ++k) sum = fmaf(__shfl(p, base + k, kWave), g - __shfl(g, base + k, kWave), sum);
    if (here) {
        dz[t * a.K + i] = live ? a.alpha * p * router_sigmoid(-z) * sum : 0.0f;
        expert[t * a.K + i] = live ? e : -1;
    }
}

// Two columns of a row at element i; n of them exist.
template <bool BF16>
__device__ __forceinline__ void load2(const void* base, int64_t i, int n, float* v) {
    if constexpr (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + i;
        v[0] = n > 0 ? bf16_bits_to_f32(p[0]) : 0.0f;
        v[1] = n > 1 ? bf16_bits_to_f32(p[1]) : 0.0f;
    } else {
        const float* p = static_cast<const float*>(base) + i;
        v[0] = n > 0 ? p[0] : 0.0f;
        v[1] = n > 1 ? p[1] : 0.0f;
    }
}

template <bool BF16>
__device__ __forceinline__ void store1(void* base, int64_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t*>(base)[i] = f32_to_bf16_bits(v);
    else static_cast<float*>(base)[i] = v;
}

// ---------------------------------------------------------------------------
// dx[t] = dx_add[t] + sum_i dz_i W[:, e_i], FP32, one rounding.  A block holds 128 columns
// of W for all experts in LDS (expert-major, 130 KB for 256 experts: one block a CU) and
// walks its tokens, a wave a token, two columns a lane: K reads of 512 bytes a token
// instead of a dense product over E.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(1024) void route_dx(RouteBackwardArgs a, int64_t per_split, const float* __restrict__ wr,
                                                 const float* __restrict__ dz, const int32_t* __restrict__ expert,
                                                 const void* dx_add, void* dx) {
    extern __shared__ float s_w[];
    const int c0 = blockIdx.x * kColTile;
    const int cols = a.H - c0 < kColTile ? a.H - c0 : kColTile;
    for (int j = threadIdx.x; j < cols * a.E; j += 1024) {
        const int c = j / a.E, e = j - c * a.E;
        s_w[e * kDxStride + c] = wr[static_cast<int64_t>(c0) * a.E + j];
    }
    __syncthreads();
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t1 = per_split * (blockIdx.y + 1) < a.T ? per_split * (blockIdx.y + 1) : a.T;
    const int c = c0 + lane * 2, n = a.H - c;
    for (int64_t t = per_split * blockIdx.y + wave; t < t1; t += 16) {
        float acc[2] = {0.0f, 0.0f};
        if (dx_add && n > 0) load2<BF16>(dx_add, t * a.H + c, n, acc);
        for (int i = 0; i < a.K; ++i) {
            const int e = expert[t * a.K + i];
            const float v = dz[t * a.K + i];
            if (e >= 0) {
                const float* w = s_w + e * kDxStride + lane * 2;
                acc[0] = fmaf(v, w[0], acc[0]);
                acc[1] = fmaf(v, w[1], acc[1]);
            }
        }
        if (n > 0) store1<BF16>(dx, t * a.H + c, acc[0]);
        if (n > 1) store1<BF16>(dx, t * a.H + c + 1, acc[1]);
    }
}

// ---------------------------------------------------------------------------
// dW[h, e] = sum_t x[t, h] dz[t, e], and the bias' gradient as column h = H with x = 1.
// A block holds the sums of 128 columns and all experts in LDS; each column belongs to one
// lane, so an LDS add meets no other lane's and the order is that of the tokens.  Token
// ranges (blockIdx.y) write partial sums.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(128) void route_dw(RouteBackwardArgs a, int64_t per_split, const void* __restrict__ x,
                                                const float* __restrict__ dz, const int32_t* __restrict__ expert,
                                                float* __restrict__ part) {
    extern __shared__ float s_acc[];
    for (int j = threadIdx.x; j < a.E * kDwStride; j += 128) s_acc[j] = 0.0f;
    __syncthreads();
    const int c0 = blockIdx.x * kColTile;
    const int col = threadIdx.x, c = c0 + col;
    const int64_t t0 = per_split * blockIdx.y;
    const int64_t t1 = t0 + per_split < a.T ? t0 + per_split : a.T;
    for (int64_t t = t0; t < t1; ++t) {
        float v = 1.0f;
        if (c < a.H) {
            if constexpr (BF16) v = bf16_bits_to_f32(static_cast<const uint16_t*>(x)[t * a.H + c]);
            else v = static_cast<const float*>(x)[t * a.H + c];
        }
        for (int i = 0; i < a.K; ++i) {
            const int e = expert[t * a.K + i];
            if (e >= 0)
                __hip_atomic_fetch_add(&s_acc[e * kDwStride + col], v * dz[t * a.K + i], __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
        }
    }
    __syncthreads();
    const int cols = a.H + 1 - c0 < kColTile ? a.H + 1 - c0 : kColTile;
    float* out = part + (static_cast<int64_t>(blockIdx.y) * (a.H + 1) + c0) * a.E;
    for (int j = threadIdx.x; j < cols * a.E; j += 128) {
        const int cc = j / a.E, e = j - cc * a.E;
        out[j] = s_acc[e * kDwStride + cc];
    }
}

// The partial sums in token order.
__global__ __launch_bounds__(256) void route_dw_sum(int64_t n, int64_t slice, int splits, int64_t bias_at,
                                                    const float* __restrict__ part, float* __restrict__ dw,
                                                    float* __restrict__ dbias) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    float v = 0.0f;
    for (int s = 0; s < splits; ++s) v += part[s * slice + i];
    if (i < bias_at) dw[i] = v;
    else if (dbias) dbias[i - bias_at] = v;
}

template <bool BF16>
static void route_backward_typed(hipStream_t st, const RouteBackwardArgs& a, const RouteBackwardPlan& p, const void* x,
                                 const float* w_router, const void* dx_add, void* dx, const float* dz,
                                 const int32_t* expert, float* part) {
    const int64_t per = (a.T + p.splits - 1) / p.splits;
    if (dx) {
        const unsigned tiles = static_cast<unsigned>((a.H + kColTile - 1) / kColTile);
        const int lds = static_cast<int>(sizeof(float)) * a.E * kDxStride;
        lds_opt_in(reinterpret_cast<const void*>(&route_dx<BF16>), sizeof(float) * kMaxExperts * kDxStride);
        route_dx<BF16><<<dim3(tiles, p.splits), 1024, lds, st>>>(a, per, w_router, dz, expert, dx_add, dx);
    }
    const unsigned tiles = static_cast<unsigned>((a.H + 1 + kColTile - 1) / kColTile);
    const int lds = static_cast<int>(sizeof(float)) * a.E * kDwStride;
    lds_opt_in(reinterpret_cast<const void*>(&route_dw<BF16>), sizeof(float) * kMaxExperts * kDwStride);
    route_dw<BF16><<<dim3(tiles, p.splits), 128, lds, st>>>(a, per, x, dz, expert, part);
}

void launch_route_backward(hipStream_t st, const RouteBackwardArgs& a, const RouteBackwardPlan& p, const void* x,
                           const float* w_router, const float* logits, const int32_t* ids, const float* dweights,
                           const void* dx_add, void* dx, float* dw_router, float* dlogit_bias, void* ws) {
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part);
    if (a.T > 0) {
        float* dz = reinterpret_cast<float*>(static_cast<char*>(ws) + p.dz);
        int32_t* expert = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + p.expert);
        int group = 1;
        while (group < a.K) group *= 2;
        route_dz<<<static_cast<unsigned>((a.T * group + 255) / 256), 256, 0, st>>>(a, group, logits, ids, dweights, dz,
                                                                                  expert);
        if (a.bf16) route_backward_typed<true>(st, a, p, x, w_router, dx_add, dx, dz, expert, part);
        else route_backward_typed<false>(st, a, p, x, w_router, dx_add, dx, dz, expert, part);
    }
    const int64_t slice = (static_cast<int64_t>(a.H) + 1) * a.E;
    route_dw_sum<<<static_cast<unsigned>((slice + 255) / 256), 256, 0, st>>>(
        slice, slice, p.splits, static_cast<int64_t>(a.H) * a.E, part, dw_router, dlogit_bias);
}

}  // namespace beam
