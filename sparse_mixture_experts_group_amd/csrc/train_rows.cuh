// Row access of the training operators: 8 consecutive columns a lane, FP32 or BF16, rows
// of any width, and the 8-bit copy (E4M3 codes, one E8M0 exponent per 32 columns).
#pragma once
#include "common.cuh"

namespace beam {

// The same 16-byte vectors at the alignment of an element: rows whose width is not a
// multiple of 8 columns start anywhere.  gfx950 loads and stores them in one instruction
// too; only the aligned forms are promised never to straddle a cache line.
typedef u32x4 u32x4_by2 __attribute__((aligned(2)));
typedef u32x4 u32x4_by4 __attribute__((aligned(4)));
typedef u32x2 u32x2_by1 __attribute__((aligned(1)));

// 8 columns as they are stored: BF16 in w[0], FP32 in w[0] and w[1].
template <bool BF16>
struct Raw8 {
    u32x4 w[BF16 ? 1 : 2];
};

// One 16-byte vector; NT: past the caches (an array that is read or written once).  4096
// tokens' sums of rows took 64 us that way, 74 through the caches.  Only aligned rows: lines
// that two vectors share are better kept (4095 tokens of 1001 FP32 columns: 22 us, 27 past
// the caches).
template <bool NT>
__device__ __forceinline__ u32x4 load_vector(const void* p) {
    return NT ? __builtin_nontemporal_load(static_cast<const u32x4*>(p)) : *static_cast<const u32x4*>(p);
}

template <bool NT>
__device__ __forceinline__ void store_vector(void* p, u32x4 v) {
    if (NT) __builtin_nontemporal_store(v, static_cast<u32x4*>(p));
    else *static_cast<u32x4*>(p) = v;
}

// Columns i .. i+7 of `base` (element index); n of them exist, the rest read as 0.
template <bool BF16, bool ALIGNED, bool NT = false>
__device__ __forceinline__ Raw8<BF16> load_raw8(const void* base, int64_t i, int n) {
    Raw8<BF16> r;
    if constexpr (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + i;
        if (ALIGNED || n >= 8) {
            r.w[0] = ALIGNED ? load_vector<NT>(p) : u32x4(*reinterpret_cast<const u32x4_by2*>(p));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = 2 * j < n ? p[2 * j] : 0, hi = 2 * j + 1 < n ? p[2 * j + 1] : 0;
                r.w[0][j] = lo | (hi << 16);
            }
        }
    } else {
        const uint32_t* p = static_cast<const uint32_t*>(base) + i;
        if (ALIGNED || n >= 8) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                r.w[k] = ALIGNED ? load_vector<NT>(p + 4 * k)
                                 : u32x4(*reinterpret_cast<const u32x4_by4*>(p + 4 * k));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r.w[j >> 2][j & 3] = j < n ? p[j] : 0;
        }
    }
    return r;
}

template <bool BF16, bool ALIGNED, bool NT = false>
__device__ __forceinline__ void store_raw8(void* base, int64_t i, int n, const Raw8<BF16>& r) {
    if constexpr (BF16) {
        uint16_t* p = static_cast<uint16_t*>(base) + i;
        if (ALIGNED) {
            store_vector<NT>(p, r.w[0]);
        } else if (n >= 8) {
            *reinterpret_cast<u32x4_by2*>(p) = r.w[0];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) p[j] = static_cast<uint16_t>(r.w[0][j >> 1] >> (16 * (j & 1)));
        }
    } else {
        uint32_t* p = static_cast<uint32_t*>(base) + i;
        if (ALIGNED) {
            store_vector<NT>(p, r.w[0]);
            store_vector<NT>(p + 4, r.w[1]);
        } else if (n >= 8) {
            *reinterpret_cast<u32x4_by4*>(p) = r.w[0];
            *reinterpret_cast<u32x4_by4*>(p + 4) = r.w[1];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) p[j] = r.w[j >> 2][j & 3];
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void widen8(const Raw8<BF16>& r, float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (BF16) v[j] = __uint_as_float((j & 1) ? (r.w[0][j >> 1] & 0xFFFF0000u) : (r.w[0][j >> 1] << 16));
        else v[j] = __uint_as_float(r.w[j >> 2][j & 3]);
    }
}

// One rounding to the stored type (BF16: to nearest even).
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> narrow8(const float* v) {
    Raw8<BF16> r;
    if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r.w[0][j] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * j])) |
                        (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * j + 1])) << 16);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j >> 2][j & 3] = __float_as_uint(v[j]);
    }
    return r;
}

// ---------------------------------------------------------------------------
// the 8-bit copy: a block of 32 columns holds E4M3 codes and one E8M0 exponent n + 127,
// value = code * 2^n, n the least integer >= -127 whose block fits: amax <= 448 * 2^n
// (448 = 1.75 * 2^8 is the largest E4M3 value).  A power of two scales without rounding,
// so a code is its value's one rounding to nearest even; the matrix cores take these
// blocks as they are.  A block that holds an infinity or a NaN gets exponent 255 (the
// E8M0 NaN) and reads back as NaN.  A lane holds 8 of the 32 columns: four lanes a block.
// ---------------------------------------------------------------------------
constexpr int kKeepBlock = 32;

__host__ __device__ inline int keep_blocks(int cols) { return (cols + kKeepBlock - 1) / kKeepBlock; }

// E8M0 code of a block from the bits of its largest magnitude.
__device__ __forceinline__ int keep_code(uint32_t amax) {
    const int ex = static_cast<int>(amax >> 23);
    const int code = ex - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return ex == 255 ? 255 : (code < 0 ? 0 : code);
}

// 2^(code - 127), NaN for 255 (2^-127 is subnormal).
__device__ __forceinline__ float keep_scale(int code) {
    const uint32_t bits = code == 0 ? 0x00400000u : static_cast<uint32_t>(code) << 23;
    return __uint_as_float(code == 255 ? 0x7fc00000u : bits);
}

// 2^(127 - code); a code that keep_code gives is at most 247, or 255 (NaN)
__device__ __forceinline__ float keep_inverse(int code) {
    return __uint_as_float(code == 255 ? 0x7fc00000u : static_cast<uint32_t>(254 - code) << 23);
}

// Encodes this lane's 8 columns with its three neighbours' (lanes 4q .. 4q+3 hold one
// block, all of them active); returns the block's exponent.  Columns that do not exist
// are passed as 0.
__device__ __forceinline__ int keep8(const float* v, u32x2& q) {
    uint32_t am = 0;                 // integer order of magnitudes: a NaN is the largest
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
        am = b > am ? b : am;
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        const uint32_t b = __shfl_xor(am, o, kWave);
        am = b > am ? b : am;
    }
    const int code = keep_code(am);
    const float inv = keep_inverse(code);
    q[0] = f32x4_to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    q[1] = f32x4_to_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    return code;
}

// 8 codes of a block with factor f.
__device__ __forceinline__ void restore8(u32x2 q, float f, float* v) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(q[k], false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(q[k], true);
        v[4 * k] = a[0] * f;
        v[4 * k + 1] = a[1] * f;
        v[4 * k + 2] = b[0] * f;
        v[4 * k + 3] = b[1] * f;
    }
}

// Factor of the block that holds column c of row r.
__device__ __forceinline__ float keep_scale_of(const uint8_t* scale, int64_t r, int cols, int c) {
    return keep_scale(scale[r * keep_blocks(cols) + c / kKeepBlock]);
}

template <bool ALIGNED, bool NT = false>
__device__ __forceinline__ u32x2 load_codes8(const uint8_t* p, int n) {
    if (ALIGNED)
        return NT ? __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p)) : *reinterpret_cast<const u32x2*>(p);
    if (n >= 8) return u32x2(*reinterpret_cast<const u32x2_by1*>(p));
    u32x2 q = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) q[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
    return q;
}

template <bool ALIGNED, bool NT = false>
__device__ __forceinline__ void store_codes8(uint8_t* p, int n, u32x2 q) {
    if (ALIGNED) {
        if (NT) __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(p));
        else *reinterpret_cast<u32x2*>(p) = q;
    } else if (n >= 8) {
        *reinterpret_cast<u32x2_by1*>(p) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = static_cast<uint8_t>(q[j >> 2] >> (8 * (j & 3)));
    }
}

// The sum of v over the `group` threads of a row, in every thread of it (a fixed tree: each
// wave's lanes, then the waves in order).  s_part: 16 floats; for a group past a wave all
// threads of the block come here together.
__device__ __forceinline__ float group_sum(float v, int group, float* s_part) {
    const int inside = group < 64 ? group : 64;
    for (int o = inside >> 1; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
    if (group > 64) {
        if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = v;
        lds_pipeline_barrier();               // waits for LDS alone, not for the row's stores
        v = 0.0f;
        for (int w = 0; w < group >> 6; ++w) v += s_part[w];
    }
    return v;
}

// Item k of a launch over pairs or, where their pairs have been written down
// (launch_invert), over rows.  `row` is where the item's values lie, -1 if nowhere; a row in
// order is read before its pair is known (`live`: whether it has one), so that no load waits
// for the look-up.  What stands in pair_of_row for a row without a pair is anything: it
// counts only if row_of_pair agrees.
struct Item {
    int64_t row, pair;
    bool live;
};
__device__ __forceinline__ Item item_at(int64_t k, int64_t pairs, int64_t rows, const int32_t* row_of_pair,
                                        const int32_t* pair_of_row) {
    Item t;
    if (pair_of_row) {
        t.row = k < rows ? k : -1;
        t.pair = k < rows ? pair_of_row[k] : -1;
        t.live = t.pair >= 0 && t.pair < pairs && row_of_pair[t.pair] == k;
    } else {
        t.pair = k;
        const int64_t r = k >= pairs ? -1 : row_of_pair ? row_of_pair[k] : k;
        t.live = r >= 0 && r < rows;
        t.row = t.live ? r : -1;
    }
    return t;
}

// Thread -> (row, 8-column piece) with rows packed back to back over the grid, so that
// narrow rows leave no lanes idle.  `pieces` per row; block b covers pieces 256 b ..
// 256 b + 255.  The division of a block's first piece is uniform; a thread's own is at
// most one more row when pieces >= 256, and exact by a 32-bit reciprocal below (numerators
// under 512).
__device__ __forceinline__ void piece_of_thread(int pieces, int64_t& row, int& piece) {
    const uint64_t first = static_cast<uint64_t>(blockIdx.x) * 256;
    const uint64_t r0 = first / static_cast<uint32_t>(pieces);
    const uint32_t at = static_cast<uint32_t>(first - r0 * static_cast<uint32_t>(pieces)) + threadIdx.x;
    const uint32_t p = static_cast<uint32_t>(pieces);
    const uint32_t more = p >= 256 ? (at >= p ? 1u : 0u) : at / p;
    row = static_cast<int64_t>(r0 + more);
    piece = static_cast<int>(at - more * p);
}

// Threads that share a row in the kernels that add over it: a lane for each 8-column piece,
// a power of two up to a wave (several rows a block of 256), or a block of whole waves (one
// row a block) of at most `most` threads, a multiple of 64 up to 1024.
inline int row_group(int cols, int most) {
    const int pieces = (cols + 7) / 8;
    if (pieces > 64) return pieces >= most ? most : (pieces + 63) / 64 * 64;
    int g = 8;
    while (g < pieces) g *= 2;
    return g;
}

// Threads that an operator has for one row, at most: a group, or the packed pieces (of whole
// blocks of the 8-bit copy).
inline int64_t row_threads(int cols) {
    const int pieces = (cols + 31) / 32 * 4, group = row_group(cols, 1024);
    return pieces > group ? pieces : group;
}

// Threads of a block, and blocks, for `rows` rows of such a group.
inline int group_threads(int group) { return group <= 64 ? 256 : group; }
inline unsigned group_blocks(int64_t rows, int group) {
    const int per = group <= 64 ? 256 / group : 1;
    return static_cast<unsigned>((rows + per - 1) / per);
}

}  // namespace beam
