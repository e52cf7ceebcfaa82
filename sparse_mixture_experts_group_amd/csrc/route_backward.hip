// Gradient of the router: from the combine weights' gradients through the normalised
// sigmoid scores to the activations, the router's weights and the logits' bias.
#include "common.cuh"
#include "kernels.h"
#include "train_kernels.h"
#include "train_rows.cuh"

namespace beam {

namespace {

constexpr int kColTile = 128;      // hidden columns of a dx block
constexpr int kDxStride = kColTile + 4;       // 16-byte rows, neighbours four banks apart
constexpr int kDwTokens = 32;      // tokens of one stage of a dW block
constexpr int kDwCols = 128;       // its hidden columns
constexpr int kBiasCols = 16;      // columns over which the bias' gradient is spread
constexpr int kCUs = 256;

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Experts of a dW block.
int dw_experts(int E) { return E <= 64 ? 64 : E <= 128 ? 128 : 256; }

// Ranges that T tokens are cut into so that `tiles` blocks a range give a CU `blocks` of
// them, a range no shorter than `least` tokens.
int token_splits(int64_t T, int64_t tiles, int blocks, int least) {
    int64_t s = blocks * kCUs / tiles;
    if (s > (T + least - 1) / least) s = (T + least - 1) / least;
    return static_cast<int>(s < 1 ? 1 : s);
}

// The bias' gradient takes part in dW's products as columns that follow the H of x: each
// stage of tokens adds to one of them in turn, and they are added up in FP64, so that its
// error stays that of the dz (one column for all: 15109 tokens and 4 experts twice that).
// Few tokens need one column.  All of them lie in one tile.
__host__ __device__ inline int bias_columns(int64_t T) { return T <= 2 * kDwTokens ? 1 : kBiasCols; }
__host__ __device__ inline int bias_first(int H, int columns) {
    return H % kDwCols + columns <= kDwCols ? H : H / kDwCols * kDwCols + kDwCols;
}

}  // namespace

RouteBackwardPlan route_backward_plan(int64_t T, int H, int E, int K) {
    RouteBackwardPlan p;
    const int bias = bias_columns(T), tiles = bias_first(H, bias) / kDwCols + 1;
    p.splits = T == 0 ? 0 : token_splits(T, tiles, 2, 2 * kDwTokens);
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off += align256(bytes); return o; };
    p.dz = take(sizeof(float) * T * K);
    p.expert = take(sizeof(int32_t) * T * K);
    p.split = take(8 * T * K);
    p.live = take(T + 8);                      // read eight at a time
    // a single range writes dW itself, and the bias' columns if they are to be added up
    p.part = take(sizeof(float) * (p.splits > 1 ? p.splits * (static_cast<size_t>(H) + bias) : bias > 1 ? bias : 0) * E);
    p.total = off;
    return p;
}

// An FP32 value as the sum of three BF16 values, 8 bits each: each remainder is exact.
__device__ __forceinline__ void split3(float v, uint16_t* s) {
    s[0] = f32_to_bf16_bits(v);
    v -= bf16_bits_to_f32(s[0]);
    s[1] = f32_to_bf16_bits(v);
    v -= bf16_bits_to_f32(s[1]);
    s[2] = f32_to_bf16_bits(v);
}

// ---------------------------------------------------------------------------
// dz: with s_i = sigma(z_i), p_i = s_i / sum_j s_j and w_i = alpha p_i,
//   dz_i = alpha p_i (1 - s_i) sum_j p_j (g_i - g_j),
// g the weights' gradients.  The sum over differences loses nothing when the g are nearly
// equal, and 1 - s_i = sigma(-z_i) nothing when s_i is near one.  A lane a pick, `group`
// lanes (a power of two, at least K) a token.  An id outside [0, E) is no pick.  Picks of
// one expert by the same token are joined in the first of them, and a token without picks
// is marked, so that what follows meets each (token, expert) once and reads no other x.
// split: a pick's dz as three BF16 values and its expert (0xFFFF: none), for dW.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void route_dz(RouteBackwardArgs a, int group, const float* __restrict__ logits,
                                                const int32_t* __restrict__ ids, const float* __restrict__ dweights,
                                                float* __restrict__ dz, int32_t* __restrict__ expert,
                                                uint16_t* __restrict__ split, uint8_t* __restrict__ alive) {
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
    const float v = live ? a.alpha * p * router_sigmoid(-z) * sum : 0.0f;
    float joined = 0.0f;
    bool first = live;
    for (int k = 0; k < a.K; ++k) {
        const bool same = __shfl(e, base + k, kWave) == e;
        joined += same ? __shfl(v, base + k, kWave) : 0.0f;
        first = first && !(same && k < i);
    }
    if (here) {
        dz[t * a.K + i] = first ? joined : 0.0f;
        expert[t * a.K + i] = first ? e : -1;
        uint16_t q[3];
        split3(joined, q);
        *reinterpret_cast<u32x2*>(split + (t * a.K + i) * 4) =
            u32x2{q[0] | (static_cast<uint32_t>(q[1]) << 16), q[2] | (first ? static_cast<uint32_t>(e) << 16 : 0xFFFF0000u)};
    }
    const uint64_t any = wave_ballot(first) >> base;
    if (here && i == 0) alive[t] = (any & ((1ull << group) - 1)) != 0;
}

// Row t of an activation array (t is the same for the whole wave: a scalar address).
template <bool BF16>
__device__ __forceinline__ const void* row_at(const void* base, int64_t t, int H) {
    return static_cast<const char*>(base) + t * H * (BF16 ? 2 : 4);
}

// Columns c, c + 1 of a row (c even) as stored: two BF16 in one word, or two FP32.  Those
// past the row come out as 0.  EVEN: H is even, so a pair lies in the row or behind it and
// is one load.  Every lane loads (clamped into the row): the loads of several rows stay in
// flight without branches between them.
template <bool BF16>
struct Pair {
    uint32_t w[BF16 ? 1 : 2];
};

template <bool BF16, bool EVEN>
__device__ __forceinline__ Pair<BF16> load2(const void* row, uint32_t H, uint32_t c) {
    Pair<BF16> p;
    if constexpr (EVEN) {
        const uint32_t at = c < H ? c / 2 : 0;
        if constexpr (BF16) {
            const uint32_t d = static_cast<const uint32_t*>(row)[at];
            p.w[0] = c < H ? d : 0;
        } else {
            const u32x2 d = static_cast<const u32x2*>(row)[at];
            p.w[0] = c < H ? d[0] : 0;
            p.w[1] = c < H ? d[1] : 0;
        }
    } else {
        const uint32_t a0 = c < H ? c : 0, a1 = c + 1 < H ? c + 1 : 0;
        if constexpr (BF16) {
            const uint32_t lo = static_cast<const uint16_t*>(row)[a0], hi = static_cast<const uint16_t*>(row)[a1];
            p.w[0] = (c < H ? lo : 0) | (c + 1 < H ? hi << 16 : 0);
        } else {
            const uint32_t lo = static_cast<const uint32_t*>(row)[a0], hi = static_cast<const uint32_t*>(row)[a1];
            p.w[0] = c < H ? lo : 0;
            p.w[1] = c + 1 < H ? hi : 0;
        }
    }
    return p;
}

// The value that lane N of this lane's row of 16 holds.
template <int N>
__device__ __forceinline__ uint32_t of_row_lane(uint32_t v) {
    return __builtin_amdgcn_update_dpp(0, v, 0x150 + N, 0xf, 0xf, true);      // row_newbcast:N
}

// The value of the next lane of the row of 16 (the last lane: of the first).
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
    return __builtin_amdgcn_update_dpp(0, v, 0x12f, 0xf, 0xf, true);          // row_ror:15
}

// ---------------------------------------------------------------------------
// dx[t] = dx_add[t] + sum_i dz_i W[:, e_i], FP32, one rounding.  A block holds 128 columns
// of W for all experts in LDS (expert-major, 130 KB for 256 experts: one block a CU) and
// walks its tokens: K reads of 512 bytes a token instead of a dense product over E.  A row
// of 16 lanes takes a token, 8 columns a lane, and holds the token's picks, a pick a lane
// (two for K > 16), which its lanes take from each other inside the vector instructions.
// The picks and addends of a wave's next tokens are loaded before it works on these.  Bound
// by HBM: 32768 tokens of 5120 BF16 columns with addends 135 us, 5.0 TB/s, 8192 in FP32 75
// us, a tenth of it W's way into LDS.  (A wave a token, two columns a lane, picks by scalar
// register: 222 us, bound by its vector instructions.)
// ---------------------------------------------------------------------------
constexpr int kDxStep = 2;         // tokens of a row of lanes in flight

template <bool BF16, bool ALIGNED, int KT, bool ADD>
__global__ __launch_bounds__(1024) void route_dx(RouteBackwardArgs a, int64_t per_split, const float* __restrict__ wr,
                                                 const float* __restrict__ dz, const int32_t* __restrict__ expert,
                                                 const void* dx_add, void* dx) {
    extern __shared__ __attribute__((aligned(16))) float s_w[];
    const int c0 = blockIdx.x * kColTile;
    static_assert(KT <= 16, "one pick a lane");
    constexpr int NP = KT > 0 ? 1 : 2;                 // picks a lane
    const int K = KT > 0 ? KT : a.K;
    const int lane = threadIdx.x & 63, in_row = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = per_split * blockIdx.y;
    const int64_t t1 = t0 + per_split < a.T ? t0 + per_split : a.T;
    const int c = c0 + in_row * 8, n = a.H - c;
    const f32x4* mine = reinterpret_cast<const f32x4*>(s_w) + in_row * 2;
    int e[kDxStep][NP], e_next[kDxStep][NP];
    float v[kDxStep][NP], v_next[kDxStep][NP];
    Raw8<BF16> add[kDxStep], add_next[kDxStep];
    auto fetch = [&](int64_t t) {                      // t: the wave's first token
#pragma unroll
        for (int s = 0; s < kDxStep; ++s) {
            const int64_t mt = t + s * 4 + (lane >> 4), at = mt < t1 ? mt : t1 - 1;
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                const int i = in_row + 16 * q;
                e_next[s][q] = expert[at * K + (i < K ? i : 0)];
                v_next[s][q] = dz[at * K + (i < K ? i : 0)];
            }
            if constexpr (ADD) {
                if (n > 0) add_next[s] = load_raw8<BF16, ALIGNED>(dx_add, at * a.H + c, n);
            }
        }
    };
    constexpr int kStride = 16 * 4 * kDxStep;          // tokens of the block's sixteen waves
    int64_t t = t0 + wave * 4 * kDxStep;
    if (t < t1) fetch(t);
    // W's columns, a wave every sixteenth: eight loads in flight
    const int cols = a.H - c0 < kColTile ? a.H - c0 : kColTile;
    for (int ee = lane; ee < a.E; ee += 64) {
        float w[kColTile / 16];
#pragma unroll
        for (int k = 0; k < kColTile / 16; ++k) {
            const int col = wave + 16 * k;
            w[k] = wr[static_cast<int64_t>(c0 + (col < cols ? col : 0)) * a.E + ee];
        }
#pragma unroll
        for (int k = 0; k < kColTile / 16; ++k) s_w[ee * kDxStride + wave + 16 * k] = w[k];
    }
    __syncthreads();
    for (; t < t1; t += kStride) {
#pragma unroll
        for (int s = 0; s < kDxStep; ++s) {
            add[s] = add_next[s];
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                // no pick: expert 0 with factor 0 (the router's weights are finite)
                e[s][q] = (e_next[s][q] > 0 ? e_next[s][q] : 0) * (kDxStride / 4);
                v[s][q] = e_next[s][q] >= 0 ? v_next[s][q] : 0.0f;
            }
        }
        if (t + kStride < t1) fetch(t + kStride);
#pragma unroll
        for (int s = 0; s < kDxStep; ++s) {
            float acc[8] = {};
            if constexpr (ADD) widen8<BF16>(add[s], acc);
            auto pick = [&](uint32_t at, uint32_t factor) {
                const float f = __uint_as_float(factor);
                const f32x4 a0 = mine[at], a1 = mine[at + 1];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[k] = fmaf(f, a0[k], acc[k]);
                    acc[4 + k] = fmaf(f, a1[k], acc[4 + k]);
                }
            };
            if constexpr (KT > 0) {
                static_for<0, KT>([&](auto i) {
                    pick(of_row_lane<i>(e[s][0]), of_row_lane<i>(__float_as_uint(v[s][0])));
                });
            } else {
                uint32_t er = e[s][0], vr = __float_as_uint(v[s][0]);
                for (int i = 0; i < K; ++i) {          // lane 0's pick, then the row moves up by one
                    if (i == 16) {
                        er = e[s][NP - 1];
                        vr = __float_as_uint(v[s][NP - 1]);
                    }
                    pick(of_row_lane<0>(er), of_row_lane<0>(vr));
                    er = row_rotate(er);
                    vr = row_rotate(vr);
                }
            }
            const int64_t mt = t + s * 4 + (lane >> 4);
            if (mt < t1 && n > 0) store_raw8<BF16, ALIGNED>(dx, mt * a.H + c, n, narrow8<BF16>(acc));
        }
    }
}

// ---------------------------------------------------------------------------
// dW[h, e] = sum_t x[t, h] dz[t, e], and the bias' gradient as columns with x = 1
// (bias_columns), on the matrix cores with the tokens as the summed index.  An FP32 value is the sum of three
// BF16 values (8 bits each, cut off by rounding to nearest: the rest is exact), so dz is
// three operands, and x is one (BF16) or three (FP32, where the six products of largest
// order are kept: the others are under 2^-24 of the result's terms).  Sums in FP32.
//
// A block: ME experts x 128 columns, four waves of 64 experts x NW columns (32 x 32 x 16
// products).  A stage of 32 tokens lies in LDS as rows of 64 bytes (one expert's operand or
// one column, 32 tokens): x is transposed in registers on its way in, dz is scattered (at
// most K entries a token) into rows that hold zeros, and its entries are taken out again
// after the products.  One buffer: two blocks share a CU (57 KB each for 256 experts and
// BF16), and one's products run while the other writes its stage.  A stage's values are
// loaded into registers a stage ahead.  Token ranges (blockIdx.y) write partial sums
// [H + bias columns, E], a single range the gradients themselves.  Matrix-bound: 32768 tokens of 5120
// columns in BF16 take 0.21 ms, 1.2 PFLOP/s of the three products, 8192 in FP32 0.115 ms,
// 1.1 of the six; a large library product in BF16 reaches 1.24.  The same sums as FP32
// additions in LDS, a lane a column, took 9.8 and 2.2 ms.
template <bool BF16, int ME, int Q_>
struct DwTile {
    static constexpr int W = 4, kThreads = W * 64;       // waves, threads
    static constexpr int WM = ME / 64, WN = W / WM;
    static constexpr int NW = kDwCols / WN, TN = NW / 32;
    static constexpr int XS = BF16 ? 1 : 3;
    static constexpr int TPW = kDwTokens / W;            // tokens whose columns a wave brings in
    static constexpr int Q = Q_;                         // picks a thread (32 K over 256 threads)
    static constexpr int kX = 3 * (ME + 1) * kStageRowBytes;         // the columns' rows
    static constexpr int kLds = kX + XS * kDwCols * kStageRowBytes;
    static_assert(TPW == 8 && kDwCols == 128, "a column's eight tokens are one 16-byte chunk, two columns a lane");
    static_assert(kLds <= 80 * 1024, "two blocks a CU");
};

// Byte of operand k of expert e, 16-byte chunk (8 tokens) `chunk`: the operands of an expert
// are neighbours; 16 experts' chunks of one product cover all banks.
__device__ __forceinline__ int dz_offset(int e, int k, int chunk) {
    return (e * 3 + k) * kStageRowBytes + ((chunk ^ ((e >> 2) & 3)) << 4);
}

template <bool BF16, bool EVEN, int ME, int Q_>
__global__ __launch_bounds__(256, 2) void route_dw(RouteBackwardArgs a, int per_split, const void* __restrict__ x,
                                                   const u32x2* __restrict__ split, const uint8_t* __restrict__ alive,
                                                   float* __restrict__ part, float* __restrict__ dw,
                                                   float* __restrict__ dbias) {
    using L = DwTile<BF16, ME, Q_>;
    extern __shared__ __attribute__((aligned(16))) char s_stage[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % L::WM, wn = wave / L::WM;
    const int c0 = blockIdx.x * kDwCols, col = lane * 2;
    const int t0 = per_split * blockIdx.y;     // T, and T * K, are below 2^30
    const int t1 = t0 + per_split < a.T ? t0 + per_split : static_cast<int>(a.T);
    for (int j = tid; j < L::kLds / 16; j += L::kThreads) reinterpret_cast<u32x4*>(s_stage)[j] = u32x4{0, 0, 0, 0};

    struct Stage {
        Pair<BF16> x[L::TPW];                  // a lane's two columns of its wave's tokens
        u32x2 live;                            // a byte each
        u32x2 pick[L::Q];                      // a thread's picks
    } ahead[2];
    const int bias = bias_columns(a.T), bias0 = bias_first(a.H, bias);
    // thread -> its picks among the stage's 32 K, and their token's place in an LDS row
    int chunk[L::Q], byte[L::Q], old[L::Q];    // old: where its picks lie in LDS
#pragma unroll
    for (int q = 0; q < L::Q; ++q) {
        const int i = tid + L::kThreads * q, tok = i < kDwTokens * a.K ? i / a.K : 0;
        chunk[q] = tok >> 3;
        byte[q] = (tok & 7) * 2;
    }
    const int end = t1 * a.K;
    // A zero that the compiler cannot tell for the same in all lanes: `alive` is then read by
    // a vector load.  A scalar one shares its counter with the LDS reads, whose waits would
    // wait for it too.
    int zero;
    asm volatile("v_mov_b32 %0, 0" : "=v"(zero));
    const uint32_t row_bytes = static_cast<uint32_t>(a.H) * (BF16 ? 2 : 4);
    auto fetch = [&](Stage& f, int t) {
        const int tw = t + wave * L::TPW, first = tw < t1 ? tw : t1 - 1, rest = t1 - 1 - first;
        // first is a multiple of 8, or past the range and of no account
        f.live = *reinterpret_cast<const u32x2*>(alive + (first & ~7) + zero);
        const char* row = static_cast<const char*>(x) + static_cast<int64_t>(first) * row_bytes;
#pragma unroll
        for (int j = 0; j < L::TPW; ++j)
            f.x[j] = load2<BF16, EVEN>(row + (j < rest ? j : rest) * row_bytes, a.H, c0 + col);
#pragma unroll
        for (int q = 0; q < L::Q; ++q) {
            const int p = t * a.K + tid + L::kThreads * q;
            f.pick[q] = split[static_cast<uint32_t>(p < end ? p : end - 1)];
        }
    };
    auto clear = [&]() {
#pragma unroll
        for (int q = 0; q < L::Q; ++q)
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<uint16_t*>(s_stage + old[q] + k * kStageRowBytes) = 0;
    };
    auto fill_dz = [&](const Stage& f, int t) {
#pragma unroll
        for (int q = 0; q < L::Q; ++q) {
            const int i = tid + L::kThreads * q, e = f.pick[q][1] >> 16;
            const bool is = i < kDwTokens * a.K && t * a.K + i < end && e != 0xFFFF;
            old[q] = dz_offset(is ? e : ME, 0, chunk[q]) + byte[q];          // none: a row of its own
            uint16_t* to = reinterpret_cast<uint16_t*>(s_stage + old[q]);
            to[0] = static_cast<uint16_t>(f.pick[q][0]);
            to[kStageRowBytes / 2] = static_cast<uint16_t>(f.pick[q][0] >> 16);
            to[kStageRowBytes] = static_cast<uint16_t>(f.pick[q][1]);
        }
    };
    auto fill_x = [&](const Stage& f, int t) {
        Pair<BF16> v[L::TPW];
#pragma unroll
        for (int j = 0; j < L::TPW; ++j) {
            // a token without picks is not looked at (live holds 0 or 1 a byte)
            const uint32_t in = t + wave * L::TPW + j < t1 ? 1 : 0;
            const uint32_t mask = 0u - ((f.live[j >> 2] >> (8 * (j & 3))) & in);
#pragma unroll
            for (int k = 0; k < (BF16 ? 1 : 2); ++k) v[j].w[k] = f.x[j].w[k] & mask;
        }
        // 1 in the stage's bias column, if it is this tile's (not asked of the others: 350 -> 340
        // us a call for 32768 tokens in BF16)
        if (c0 + kDwCols > a.H) {
            const int one = bias0 + ((t / kDwTokens) & (bias - 1)) - c0 - col;
#pragma unroll
            for (int j = 0; j < L::TPW; ++j) {
                if constexpr (BF16) {
                    v[j].w[0] |= one == 0 ? 0x3F80u : one == 1 ? 0x3F800000u : 0u;
                } else {
                    v[j].w[0] |= one == 0 ? 0x3F800000u : 0u;
                    v[j].w[1] |= one == 1 ? 0x3F800000u : 0u;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {          // a column: the wave's eight tokens, a chunk
            char* to = s_stage + L::kX + stage_offset(col + k, wave);
            if constexpr (BF16) {
                const uint32_t sel = k == 0 ? 0x05040100u : 0x07060302u;          // low or high halves
                u32x4 o;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = __builtin_amdgcn_perm(v[2 * j + 1].w[0], v[2 * j].w[0], sel);
                *reinterpret_cast<u32x4*>(to) = o;
            } else {
                uint16_t p[L::TPW][3];
#pragma unroll
                for (int j = 0; j < L::TPW; ++j) split3(__uint_as_float(v[j].w[k]), p[j]);
#pragma unroll
                for (int m = 0; m < 3; ++m) {
                    u32x4 o;
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = p[2 * j][m] | (static_cast<uint32_t>(p[2 * j + 1][m]) << 16);
                    *reinterpret_cast<u32x4*>(to + m * kDwCols * kStageRowBytes) = o;
                }
            }
        }
    };

    f32x16 acc[2][L::TN] = {};
    struct Operands {
        bf16x8 z[2][3], x[L::TN][L::XS];
    };
    auto read = [&](Operands& f, int ks) {
        const int ch = ks * 2 + (lane >> 5);
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                f.z[i][k] =
                    *reinterpret_cast<const bf16x8*>(s_stage + dz_offset(wm * 64 + i * 32 + (lane & 31), k, ch));
#pragma unroll
        for (int k = 0; k < L::XS; ++k)
#pragma unroll
            for (int i = 0; i < L::TN; ++i)
                f.x[i][k] = *reinterpret_cast<const bf16x8*>(s_stage + L::kX + k * kDwCols * kStageRowBytes +
                                                             stage_offset(wn * L::NW + i * 32 + (lane & 31), ch));
    };
    auto multiply = [&](const Operands& f) {
#pragma unroll
        for (int order = 2; order >= 0; --order)         // small products first
#pragma unroll
            for (int k = 0; k < L::XS; ++k)
                if (order - k >= 0) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < L::TN; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.z[i][order - k], f.x[j][k], acc[i][j],
                                                                               0, 0, 0);
                }
    };
    auto products = [&]() {
        if constexpr (L::XS == 1 && L::Q == 1) {
            // the second half's operands come between the first half's matrix instructions;
            // with more operands or picks there are not the registers for both
            constexpr int NR = 6 + L::TN, NM = 2 * L::TN * 3;
            Operands f[2];
            __builtin_amdgcn_sched_barrier(0);
            read(f[0], 0);
            read(f[1], 1);
            multiply(f[0]);
            multiply(f[1]);
            __builtin_amdgcn_sched_group_barrier(0x100, NR, 0);
            static_for<0, 2 * NM>([](auto i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if constexpr (i < NR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            });
            __builtin_amdgcn_sched_barrier(0);
        } else {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Operands f;
                read(f, ks);
                multiply(f);
            }
        }
    };

    __syncthreads();
    if (t0 < t1) {
        fetch(ahead[0], t0);
        fetch(ahead[1], t0 + kDwTokens);
        fill_x(ahead[0], t0);
        fill_dz(ahead[0], t0);
    }
    // pairs of stages, the last one perhaps empty
    for (int t = t0; t < t1; t += 2 * kDwTokens) {
        static_for<0, 2>([&](auto u) {
            const int tu = t + u * kDwTokens;
            lds_pipeline_barrier();            // the stage is written
            fetch(ahead[u], tu + 2 * kDwTokens);
            products();
            lds_pipeline_barrier();            // and read
            clear();
            fill_x(ahead[u ^ 1], tu + kDwTokens);
            lds_pipeline_barrier();            // no entry of it is left
            fill_dz(ahead[u ^ 1], tu + kDwTokens);
        });
    }

    // lane: column n = lane % 32 of its tile, experts 8 (r / 4) + 4 (lane / 32) + r % 4
#pragma unroll
    for (int j = 0; j < L::TN; ++j) {
        const int c = c0 + wn * L::NW + j * 32 + (lane & 31);
        const int b = c - bias0;               // a bias column if in [0, bias)
        if (c >= a.H && (b < 0 || b >= bias)) continue;
        float* out;
        if (gridDim.y > 1) out = part + (static_cast<int64_t>(blockIdx.y) * (a.H + bias) + (c < a.H ? c : a.H + b)) * a.E;
        else if (c < a.H) out = dw + static_cast<int64_t>(c) * a.E;
        else out = bias > 1 ? part + b * a.E : dbias;
        if (!out) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int e = wm * 64 + i * 32 + 2 * r + 4 * (lane >> 5);
                const f32x4 v = {acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
                if (a.E % 4 == 0) {
                    if (e < a.E) *reinterpret_cast<f32x4*>(out + e) = v;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (e + k < a.E) out[e + k] = v[k];
                }
            }
    }
}

// The partial sums in token order, eight loads in flight (with one, 9021 tokens of 128 columns
// and 3 experts took 49 us a call, not 26): blocks of 256 values of dW, `blocks` of them,
// then blocks of 16 experts' bias, a thread a column and expert, in FP64.
__global__ __launch_bounds__(256) void route_dw_sum(int64_t n, int64_t slice, int splits, unsigned blocks, int E,
                                                    int bias, int64_t bias_at, const float* __restrict__ part,
                                                    float* __restrict__ dw, float* __restrict__ dbias) {
    if (blockIdx.x < blocks) {
        const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
        if (i >= n) return;
        float v = 0.0f;
#pragma unroll 8
        for (int s = 0; s < splits; ++s) v += part[s * slice + i];
        dw[i] = v;
        return;
    }
    static_assert(kBiasCols == 16, "256 threads are 16 columns of 16 experts");
    __shared__ double s_sum[kBiasCols][16];
    const int b = threadIdx.x >> 4, k = threadIdx.x & 15;
    const int e = static_cast<int>(blockIdx.x - blocks) * 16 + k;
    double v = 0.0;
    if (b < bias && e < E) {
#pragma unroll 8
        for (int s = 0; s < splits; ++s) v += part[s * slice + bias_at + b * E + e];
    }
    s_sum[b][k] = v;
    __syncthreads();
    if (b == 0 && e < E) {
        for (int j = 1; j < bias; ++j) v += s_sum[j][k];
        dbias[e] = static_cast<float>(v);
    }
}

template <bool BF16, bool ALIGNED, int KT>
static void dx_launch(hipStream_t st, const RouteBackwardArgs& a, const float* w_router, const float* dz,
                      const int32_t* expert, const void* dx_add, void* dx) {
    const int tiles = (a.H + kColTile - 1) / kColTile;
    const int splits = token_splits(a.T, tiles, 1, 64);
    const int64_t per = (a.T + splits - 1) / splits;
    const auto kernel = dx_add ? &route_dx<BF16, ALIGNED, KT, true> : &route_dx<BF16, ALIGNED, KT, false>;
    lds_opt_in(reinterpret_cast<const void*>(kernel), sizeof(float) * kMaxExperts * kDxStride);
    kernel<<<dim3(tiles, splits), 1024, sizeof(float) * a.E * kDxStride, st>>>(a, per, w_router, dz, expert, dx_add, dx);
}

template <bool BF16, bool EVEN, int ME, int Q>
static void dw_launch_picks(hipStream_t st, const RouteBackwardArgs& a, int splits, const void* x, const u32x2* split,
                            const uint8_t* alive, float* part, float* dw, float* dbias) {
    using L = DwTile<BF16, ME, Q>;
    const int per = static_cast<int>(((a.T + splits - 1) / splits + kDwTokens - 1) / kDwTokens * kDwTokens);
    lds_opt_in(reinterpret_cast<const void*>(&route_dw<BF16, EVEN, ME, Q>), L::kLds);
    route_dw<BF16, EVEN, ME, Q><<<dim3(bias_first(a.H, bias_columns(a.T)) / kDwCols + 1, splits), L::kThreads, L::kLds, st>>>(
        a, per, x, split, alive, part, dw, dbias);
}

template <bool BF16, bool EVEN, int ME>
static void dw_launch(hipStream_t st, const RouteBackwardArgs& a, int splits, const void* x, const u32x2* split,
                      const uint8_t* alive, float* part, float* dw, float* dbias) {
    if (a.K <= 8) dw_launch_picks<BF16, EVEN, ME, 1>(st, a, splits, x, split, alive, part, dw, dbias);
    else dw_launch_picks<BF16, EVEN, ME, 4>(st, a, splits, x, split, alive, part, dw, dbias);
}

template <bool BF16, bool EVEN>
static void route_backward_typed(hipStream_t st, const RouteBackwardArgs& a, const RouteBackwardPlan& p, const void* x,
                                 const float* w_router, const void* dx_add, void* dx, const float* dz,
                                 const int32_t* expert, const u32x2* split, const uint8_t* alive, float* part,
                                 float* dw, float* dbias) {
    if (dx) {
        const bool al = a.H % 8 == 0;
        if (al && a.K == 8) dx_launch<BF16, true, 8>(st, a, w_router, dz, expert, dx_add, dx);
        else if (al) dx_launch<BF16, true, 0>(st, a, w_router, dz, expert, dx_add, dx);
        else dx_launch<BF16, false, 0>(st, a, w_router, dz, expert, dx_add, dx);
    }
    const int me = dw_experts(a.E);
    if (me == 64) dw_launch<BF16, EVEN, 64>(st, a, p.splits, x, split, alive, part, dw, dbias);
    else if (me == 128) dw_launch<BF16, EVEN, 128>(st, a, p.splits, x, split, alive, part, dw, dbias);
    else dw_launch<BF16, EVEN, 256>(st, a, p.splits, x, split, alive, part, dw, dbias);
}

void launch_route_backward(hipStream_t st, const RouteBackwardArgs& a, const RouteBackwardPlan& p, const void* x,
                           const float* w_router, const float* logits, const int32_t* ids, const float* dweights,
                           const void* dx_add, void* dx, float* dw_router, float* dlogit_bias, void* ws) {
    char* base = static_cast<char*>(ws);
    float* part = reinterpret_cast<float*>(base + p.part);
    if (a.T > 0) {
        float* dz = reinterpret_cast<float*>(base + p.dz);
        int32_t* expert = reinterpret_cast<int32_t*>(base + p.expert);
        uint16_t* split = reinterpret_cast<uint16_t*>(base + p.split);
        uint8_t* alive = reinterpret_cast<uint8_t*>(base + p.live);
        int group = 1;
        while (group < a.K) group *= 2;
        route_dz<<<static_cast<unsigned>((a.T * group + 255) / 256), 256, 0, st>>>(a, group, logits, ids, dweights, dz,
                                                                                  expert, split, alive);
        const bool even = a.H % 2 == 0;
        const auto run = a.bf16 ? (even ? &route_backward_typed<true, true> : &route_backward_typed<true, false>)
                                : (even ? &route_backward_typed<false, true> : &route_backward_typed<false, false>);
        run(st, a, p, x, w_router, dx_add, dx, dz, expert, reinterpret_cast<const u32x2*>(split), alive, part,
            dw_router, dlogit_bias);
    }
    const int bias = bias_columns(a.T);
    const int64_t values = p.splits == 1 ? 0 : static_cast<int64_t>(a.H) * a.E;      // of dW, to add up
    const unsigned blocks = static_cast<unsigned>((values + 255) / 256);
    const unsigned bias_blocks = dlogit_bias && (p.splits != 1 || bias > 1) ? (a.E + 15) / 16 : 0;
    if (blocks + bias_blocks == 0) return;
    route_dw_sum<<<blocks + bias_blocks, 256, 0, st>>>(values, values + static_cast<int64_t>(bias) * a.E, p.splits,
                                                       blocks, a.E, bias, values, part, dw_router, dlogit_bias);
}

}  // namespace beam
