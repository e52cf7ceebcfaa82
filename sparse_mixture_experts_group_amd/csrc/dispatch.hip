// Tokens sorted by expert, copied into rows and added up again, with gradients.
#include "common.cuh"
#include "kernels.h"
#include "train_kernels.h"
#include "train_rows.cuh"

namespace beam {

// ---------------------------------------------------------------------------
// sort: row(p) = #{q : e_q < e_p} + #{q < p : e_q = e_p} over the pairs whose expert id
// lies in [0, E); other pairs are dropped (row -1).  A counting sort: integer counts,
// so every order of the additions gives the same rows.
// ---------------------------------------------------------------------------
// Lanes of the wave that hold the same expert id as this one (ids below 256), among the
// lanes of `valid`: one ballot per id bit.
__device__ __forceinline__ uint64_t same_expert(int e, uint64_t valid) {
    uint64_t m = valid;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint64_t set = wave_ballot((e >> b) & 1);
        m &= ((e >> b) & 1) ? set : ~set;
    }
    return m;
}

// Counts of a chunk's experts (256 of them; those past E stay 0).
__global__ __launch_bounds__(256) void sort_count(int64_t pairs, int64_t chunk, int E, const int32_t* __restrict__ ids,
                                                  int32_t* __restrict__ counts) {
    __shared__ int s_cnt[kMaxExperts];
    s_cnt[threadIdx.x] = 0;
    __syncthreads();
    const int64_t p0 = chunk * blockIdx.x, p1 = p0 + chunk < pairs ? p0 + chunk : pairs;
    for (int64_t p = p0 + threadIdx.x; p < p1; p += 256) {
        const int e = ids[p];
        if (e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
    }
    __syncthreads();
    counts[blockIdx.x * kMaxExperts + threadIdx.x] = s_cnt[threadIdx.x];
}

// Exclusive prefix sum over the first 256 threads' values (thread order), and the total.
// Every thread of the block calls it; sh holds 4 ints.
__device__ __forceinline__ int scan256(int v, int* sh, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o, kWave);
        if (lane >= o) x += y;
    }
    if (lane == 63 && wave < 4) sh[wave] = x;
    __syncthreads();
    int before = 0, tot = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int t = sh[w];
        before += w < wave ? t : 0;
        tot += t;
    }
    __syncthreads();
    total = tot;
    return before + x - v;
}

// Ranks and writes one chunk.  Each of the NW waves owns a contiguous part of it: counts
// of its part first, then, with the offsets of the chunks and waves before it, each group of
// 64 pairs in order (rank inside the group from same_expert).  SINGLE: the chunk is the
// batch, and the expert offsets come from its own counts; otherwise every block adds up all
// chunks' counts (at most 256 KB out of L2) rather than wait for another launch.
template <int NW, bool SINGLE>
__global__ __launch_bounds__(NW * 64) void sort_scatter(int64_t pairs, int64_t chunk, int E,
                                                        const int32_t* __restrict__ ids,
                                                        const int32_t* __restrict__ counts,
                                                        int32_t* __restrict__ expert_off,
                                                        int32_t* __restrict__ row_of_pair,
                                                        int32_t* __restrict__ pair_of_row) {
    static_assert(NW >= 4, "a thread an expert");
    __shared__ int s_at[NW][kMaxExperts];     // counts, then the next row, per wave and expert
    __shared__ __attribute__((aligned(16))) int s_all[SINGLE ? 1 : 2 * NW][kMaxExperts];
    __shared__ int sh[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t p0 = SINGLE ? 0 : chunk * blockIdx.x;
    const int64_t n = SINGLE ? pairs : (pairs - p0 < chunk ? pairs - p0 : chunk);
    const int64_t part = ((n + NW - 1) / NW + 63) / 64 * 64;
    const int64_t lo = wave * part, hi = lo + part < n ? lo + part : n;
    for (int i = tid; i < NW * kMaxExperts; i += NW * 64) s_at[0][i] = 0;
    if constexpr (!SINGLE) {                  // a lane four experts, a wave every NWth chunk
        typedef int i32x4 __attribute__((ext_vector_type(4)));
        i32x4 before = {0, 0, 0, 0}, all = {0, 0, 0, 0};
        const int nblk = gridDim.x;
#pragma unroll 8
        for (int b = wave; b < nblk; b += NW) {
            const i32x4 v = *reinterpret_cast<const i32x4*>(counts + b * kMaxExperts + lane * 4);
            all += v;
            before += b < static_cast<int>(blockIdx.x) ? v : i32x4{0, 0, 0, 0};
        }
        *reinterpret_cast<i32x4*>(&s_all[wave][lane * 4]) = all;
        *reinterpret_cast<i32x4*>(&s_all[NW + wave][lane * 4]) = before;
    }
    __syncthreads();
    for (int64_t j = lo + lane; j < hi; j += 64) {
        const int e = ids[p0 + j];
        if (e >= 0 && e < E) atomicAdd(&s_at[wave][e], 1);
    }
    __syncthreads();
    int count = 0, at = 0;
    if (tid < E) {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            count += SINGLE ? s_at[w][tid] : s_all[w][tid];
            if constexpr (!SINGLE) at += s_all[NW + w][tid];
        }
    }
    int live;                                 // rows in all
    const int off = scan256(count, sh, live);
    if (tid < E) {
        at += off;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const int c = s_at[w][tid];
            s_at[w][tid] = at;
            at += c;
        }
        if (blockIdx.x == 0) expert_off[tid] = off;
    }
    if (blockIdx.x == 0 && tid == 0) expert_off[E] = live;
    __syncthreads();
    for (int64_t j0 = lo; j0 < hi; j0 += 64) {    // wave-uniform bounds
        const int64_t j = j0 + lane;
        const int e = j < hi ? ids[p0 + j] : -1;
        const bool ok = e >= 0 && e < E;
        const uint64_t same = same_expert(e, wave_ballot(ok));
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        if (ok) {
            const int row = s_at[wave][e] + rank;
            row_of_pair[p0 + j] = row;
            pair_of_row[row] = static_cast<int32_t>(p0 + j);
        } else if (j < hi) {
            row_of_pair[p0 + j] = -1;
        }
        __builtin_amdgcn_wave_barrier();      // every lane has read its offset
        if (ok && (same >> lane) == 1) s_at[wave][e] += rank + 1;      // the last of its kind
        __builtin_amdgcn_wave_barrier();
    }
    // rows behind the last one belong to no pair
    for (int64_t j = tid; j < n; j += NW * 64)
        if (p0 + j >= live) pair_of_row[p0 + j] = -1;
}

void launch_sort_pairs(hipStream_t st, int64_t pairs, int E, const int32_t* ids, int32_t* expert_off,
                       int32_t* row_of_pair, int32_t* pair_of_row, int32_t* counts) {
    const int64_t nblk = sort_blocks(pairs);
    if (nblk == 0) {
        // a few pairs need no sixteen waves' counters
        if (pairs <= 512)
            sort_scatter<4, true><<<1, 256, 0, st>>>(pairs, 0, E, ids, nullptr, expert_off, row_of_pair, pair_of_row);
        else
            sort_scatter<16, true><<<1, 1024, 0, st>>>(pairs, 0, E, ids, nullptr, expert_off, row_of_pair, pair_of_row);
        return;
    }
    const int64_t chunk = sort_chunk(pairs);
    sort_count<<<static_cast<unsigned>(nblk), 256, 0, st>>>(pairs, chunk, E, ids, counts);
    sort_scatter<4, false><<<static_cast<unsigned>(nblk), 256, 0, st>>>(pairs, chunk, E, ids, counts, expert_off,
                                                                        row_of_pair, pair_of_row);
}

// pair_of_row for operators that take rows in order: one stream of addresses an array,
// instead of one an expert, is worth this pass of 8 bytes a pair where rows_in_order says so.
__global__ __launch_bounds__(256) void invert_rows(int64_t pairs, int64_t rows, const int32_t* __restrict__ row_of_pair,
                                                   int32_t* __restrict__ pair_of_row, float* __restrict__ dweights) {
    const int64_t p = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (p >= pairs) return;
    const int64_t r = row_of_pair[p];
    if (r >= 0 && r < rows) pair_of_row[r] = static_cast<int32_t>(p);
    else if (dweights) dweights[p] = 0.0f;
}

void launch_invert(hipStream_t st, int64_t pairs, int64_t rows, const int32_t* row_of_pair, int32_t* pair_of_row,
                   float* dweights) {
    invert_rows<<<static_cast<unsigned>((pairs + 255) / 256), 256, 0, st>>>(pairs, rows, row_of_pair, pair_of_row,
                                                                           dweights);
}

// ---------------------------------------------------------------------------
// dispatch: xs[row_i] = x[t].  Each 8-column piece of a token is read once and written to
// its K rows; with KEEP the 8-bit copy of x leaves in the same pass.  Bound by HBM writes:
// 32768 skewed tokens of 5120 BF16 columns with the copy, 3.2 GB, take 0.55 ms (5.7 TB/s);
// 8192 tokens out of the copy 134 us (5.3).  A thread a written piece reads x through the L2
// of every XCD: 0.98 ms.  Two or four pieces a thread, and stores past the caches, spread
// the rows in flight: 0.61, 0.65 and 0.59 ms.
// ---------------------------------------------------------------------------
// Row of pick i of token t, or -1 if it has none in the buffer.
__device__ __forceinline__ int64_t row_of(const RowArgs& a, int64_t t, int i) {
    const int64_t r = a.row_of_pair ? a.row_of_pair[t * a.K + i] : t;
    return r >= 0 && r < a.rows ? r : -1;
}

template <bool BF16, bool ALIGNED, bool SRC8, bool KEEP>
__global__ __launch_bounds__(256) void dispatch_rows(RowArgs a, int pieces, const void* __restrict__ x,
                                                     const uint8_t* __restrict__ x_scale, void* __restrict__ xs,
                                                     uint8_t* __restrict__ keep_q, uint8_t* __restrict__ keep_scale) {
    int64_t t;
    int piece;
    piece_of_thread(pieces, t, piece);
    const int c = piece * 8, n = a.H - c;
    const bool here = t < a.T && n > 0;
    Raw8<BF16> v = {};
    if (here) {
        if constexpr (SRC8) {
            const u32x2 q = load_codes8<ALIGNED>(static_cast<const uint8_t*>(x) + t * a.H + c, n);
            float f[8];
            restore8(q, keep_scale_of(x_scale, t, a.H, c), f);
            v = narrow8<BF16>(f);
        } else {
            v = load_raw8<BF16, ALIGNED>(x, t * a.H + c, n);
        }
    }
    if constexpr (KEEP) {                     // all lanes: four of them share a block
        float f[8];
        widen8<BF16>(v, f);
        u32x2 q;
        const int code = keep8(f, q);
        if (here) {
            store_codes8<ALIGNED>(keep_q + t * a.H + c, n, q);
            if ((piece & 3) == 0) keep_scale[t * keep_blocks(a.H) + piece / 4] = static_cast<uint8_t>(code);
        }
    }
    if (!here || !xs) return;
    for (int i0 = 0; i0 < a.K; i0 += 8) {
        int64_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = i0 + j < a.K ? row_of(a, t, i0 + j) : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (r[j] >= 0) store_raw8<BF16, ALIGNED>(xs, r[j] * a.H + c, n, v);
    }
}

// Blocks of 256 threads over `rows` rows of `pieces` pieces.
static unsigned piece_blocks(int64_t rows, int pieces) {
    return static_cast<unsigned>((rows * pieces + 255) / 256);
}

template <bool BF16, bool ALIGNED>
static void dispatch_typed(hipStream_t st, const RowArgs& a, const void* x, const uint8_t* x_scale, void* xs,
                           uint8_t* keep_q, uint8_t* keep_scale) {
    int pieces = (a.H + 7) / 8;
    if (keep_q) {
        pieces = (pieces + 3) / 4 * 4;        // whole blocks of four lanes
        dispatch_rows<BF16, ALIGNED, false, true><<<piece_blocks(a.T, pieces), 256, 0, st>>>(
            a, pieces, x, nullptr, xs, keep_q, keep_scale);
    } else if (x_scale) {
        dispatch_rows<BF16, ALIGNED, true, false><<<piece_blocks(a.T, pieces), 256, 0, st>>>(
            a, pieces, x, x_scale, xs, nullptr, nullptr);
    } else {
        dispatch_rows<BF16, ALIGNED, false, false><<<piece_blocks(a.T, pieces), 256, 0, st>>>(
            a, pieces, x, nullptr, xs, nullptr, nullptr);
    }
}

void launch_dispatch(hipStream_t st, const RowArgs& a, const void* x, const uint8_t* x_scale, void* xs,
                     uint8_t* keep_q, uint8_t* keep_scale) {
    if (a.T == 0) return;
    const bool al = a.H % 8 == 0;
    if (a.bf16 && al) dispatch_typed<true, true>(st, a, x, x_scale, xs, keep_q, keep_scale);
    else if (a.bf16) dispatch_typed<true, false>(st, a, x, x_scale, xs, keep_q, keep_scale);
    else if (al) dispatch_typed<false, true>(st, a, x, x_scale, xs, keep_q, keep_scale);
    else dispatch_typed<false, false>(st, a, x, x_scale, xs, keep_q, keep_scale);
}

// ---------------------------------------------------------------------------
// combine: y[t] = sum_i w_i in[row_i], i ascending, FP32, one rounding at the end; dropped
// picks are not read and add nothing (a token without rows gets zeros).  Without weights
// this is the gradient of dispatch.  Bound by HBM reads, each byte once and eight loads in
// flight a thread: 4096 tokens of 5120 BF16 columns 64 us (5.9 TB/s), 4095 of 1001 FP32
// columns 22 us (5.0; rows that start anywhere).
// ---------------------------------------------------------------------------
template <bool BF16, bool ALIGNED>
__global__ __launch_bounds__(256) void combine_rows(RowArgs a, int pieces, const void* __restrict__ in,
                                                    void* __restrict__ y) {
    int64_t t;
    int piece;
    piece_of_thread(pieces, t, piece);
    const int c = piece * 8, n = a.H - c;
    if (t >= a.T) return;
    float acc[8] = {};
    for (int i0 = 0; i0 < a.K; i0 += 8) {
        int64_t r[8];
        float w[8];
        Raw8<BF16> v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = i0 + j < a.K ? row_of(a, t, i0 + j) : -1;
            w[j] = i0 + j < a.K && a.weights ? a.weights[t * a.K + i0 + j] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (r[j] >= 0) v[j] = load_raw8<BF16, ALIGNED, true>(in, r[j] * a.H + c, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (r[j] >= 0) {
                float f[8];
                widen8<BF16>(v[j], f);
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = fmaf(w[j], f[k], acc[k]);
            }
        }
    }
    store_raw8<BF16, ALIGNED, true>(y, t * a.H + c, n, narrow8<BF16>(acc));
}

void launch_combine_rows(hipStream_t st, const RowArgs& a, const void* in, void* y) {
    if (a.T == 0) return;
    const int pieces = (a.H + 7) / 8;
    const unsigned blocks = piece_blocks(a.T, pieces);
    const bool al = a.H % 8 == 0;
    if (a.bf16 && al) combine_rows<true, true><<<blocks, 256, 0, st>>>(a, pieces, in, y);
    else if (a.bf16) combine_rows<true, false><<<blocks, 256, 0, st>>>(a, pieces, in, y);
    else if (al) combine_rows<false, true><<<blocks, 256, 0, st>>>(a, pieces, in, y);
    else combine_rows<false, false><<<blocks, 256, 0, st>>>(a, pieces, in, y);
}

// ---------------------------------------------------------------------------
// gradient of combine: deo[row_i] = w_i dy[t], dw[t, i] = <dy[t], eo[row_i]>.  A group of
// threads shares a token (row_group): each piece of dy is read once for all picks, the K
// dot products are kept in FP32 registers and added over the group at the end.  A thread
// writes deo where it has read eo, so the two may be one buffer.  Bound by HBM over as many
// streams as experts: 8192 tokens of 5120 BF16 columns 268 us (5.3 TB/s).  In the order of
// rows (one stream each, as the SwiGLU) dy is read K times over: 365 us.
// ---------------------------------------------------------------------------
template <bool BF16, bool ALIGNED, bool DOT, int P>
__global__ __launch_bounds__(1024) void combine_backward(RowArgs a, int group, const void* __restrict__ dy,
                                                         const void* eo, void* deo, float* __restrict__ dweights) {
    __shared__ float s_dot[P][16];
    const int lane = group <= 64 ? threadIdx.x & (group - 1) : threadIdx.x;
    const int64_t t = group <= 64 ? static_cast<int64_t>(blockIdx.x) * (256 / group) + threadIdx.x / group : blockIdx.x;
    const bool here = t < a.T;
    for (int i0 = 0; i0 < a.K; i0 += P) {
        int64_t r[P];
        float w[P], dot[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            r[j] = here && i0 + j < a.K ? row_of(a, t, i0 + j) : -1;
            w[j] = r[j] >= 0 ? a.weights[t * a.K + i0 + j] : 1.0f;
            dot[j] = 0.0f;
        }
        if (here) {
            for (int c = lane * 8; c < a.H; c += group * 8) {
                const int n = a.H - c;
                float g[8];
                widen8<BF16>(load_raw8<BF16, ALIGNED>(dy, t * a.H + c, n), g);
                Raw8<BF16> v[P];
                if constexpr (DOT) {
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        if (r[j] >= 0) v[j] = load_raw8<BF16, ALIGNED, true>(eo, r[j] * a.H + c, n);
                }
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (r[j] >= 0) {
                        float o[8];
                        if constexpr (DOT) {
                            float f[8];
                            widen8<BF16>(v[j], f);
#pragma unroll
                            for (int k = 0; k < 8; ++k) dot[j] = fmaf(g[k], f[k], dot[j]);
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = w[j] * g[k];
                        store_raw8<BF16, ALIGNED, true>(deo, r[j] * a.H + c, n, narrow8<BF16>(o));
                    }
                }
            }
        }
        if constexpr (DOT) {
            // the barriers wait for LDS alone, not for deo's stores
            if (i0 > 0 && group > 64) lds_pipeline_barrier();        // the last picks' sums have been read
            // wave sums of all picks, one meeting of the waves, then a thread a pick adds
            // them in wave order
            const int inside = group < 64 ? group : 64;
#pragma unroll
            for (int j = 0; j < P; ++j)
                for (int o = inside >> 1; o >= 1; o >>= 1) dot[j] += __shfl_xor(dot[j], o, kWave);
            if (group > 64) {
                if ((threadIdx.x & 63) == 0) {
#pragma unroll
                    for (int j = 0; j < P; ++j) s_dot[j][threadIdx.x >> 6] = dot[j];
                }
                lds_pipeline_barrier();
                if (here && lane < P && i0 + lane < a.K) {
                    float sum = 0.0f;
                    for (int v = 0; v < group >> 6; ++v) sum += s_dot[lane][v];
                    dweights[t * a.K + i0 + lane] = sum;      // 0 for a dropped pick
                }
            } else if (here && lane == 0) {
#pragma unroll
                for (int j = 0; j < P; ++j)
                    if (i0 + j < a.K) dweights[t * a.K + i0 + j] = dot[j];
            }
        }
    }
}

template <bool BF16, bool ALIGNED, int P>
static void combine_backward_picks(hipStream_t st, const RowArgs& a, int group, const void* dy, const void* eo,
                                   void* deo, float* dweights) {
    const unsigned blocks = group_blocks(a.T, group);
    const int threads = group_threads(group);
    if (eo) combine_backward<BF16, ALIGNED, true, P><<<blocks, threads, 0, st>>>(a, group, dy, eo, deo, dweights);
    else combine_backward<BF16, ALIGNED, false, P><<<blocks, threads, 0, st>>>(a, group, dy, nullptr, deo, nullptr);
}

// P picks at a time, 32 registers of eo at most.  Of BF16 fewer where there are fewer picks:
// the waves then need half the registers, and twice as many are there to wait for memory.
// 4096 tokens of 5120 BF16 columns: two picks 36 us at two at a time, 45 at eight; four 68
// at four, 71 at eight.  FP32 stays at four: two picks 78 us, at two at a time 82.
template <bool BF16, bool ALIGNED>
static void combine_backward_typed(hipStream_t st, const RowArgs& a, int group, const void* dy, const void* eo,
                                   void* deo, float* dweights) {
    if constexpr (BF16) {
        if (a.K <= 2) return combine_backward_picks<BF16, ALIGNED, 2>(st, a, group, dy, eo, deo, dweights);
        if (a.K > 4) return combine_backward_picks<BF16, ALIGNED, 8>(st, a, group, dy, eo, deo, dweights);
    }
    combine_backward_picks<BF16, ALIGNED, 4>(st, a, group, dy, eo, deo, dweights);
}

void launch_combine_backward(hipStream_t st, const RowArgs& a, const void* dy, const void* eo, void* deo,
                             float* dweights) {
    if (a.T == 0) return;
    // 8192 tokens of 5120 columns: 269 us with 64 to 256 threads a token (5.3 TB/s), 277 with
    // 320, 309 with 640; a few tokens want more threads each
    const int group = row_group(a.H, 256);
    const bool al = a.H % 8 == 0;
    if (a.bf16 && al) combine_backward_typed<true, true>(st, a, group, dy, eo, deo, dweights);
    else if (a.bf16) combine_backward_typed<true, false>(st, a, group, dy, eo, deo, dweights);
    else if (al) combine_backward_typed<false, true>(st, a, group, dy, eo, deo, dweights);
    else combine_backward_typed<false, false>(st, a, group, dy, eo, deo, dweights);
}

}  // namespace beam
