// kvx_dense.hpp -- dense rows and pools of other types: rows quantised to 4 bits
// as they are written, and rows of a pool read back (gfx950 / CDNA4).
//
// A block of 32 values x, y = x / scale, takes the power of two
//   2^e, e = min {e : max |y| <= 7 * 2^e} held inside -23 .. 13,
// and its numbers are the nearest e2m1 values of y / 2^e (even on a tie, 6 past
// it).  7 and not 6: a largest value between 6 and 7 is off by at most 1 * 2^e,
// as it would be under 2^(e+1), and the others keep the finer step.  The bounds
// make every held value a multiple of 2^-24 of at most 49152, which f16, bf16
// and f32 all have exactly: reading rounds only where a scale is multiplied.
#pragma once

#include "kvx_tables.hpp"

namespace kvx {
namespace tables {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kBlockBase = 127;         // a scale byte s stands for 2^(s - kBlockBase)
constexpr uint32_t kLeastBlock = kBlockBase - 23, kMostBlock = kBlockBase + 13;
constexpr uint32_t kNanBlock = 255;

struct DenseArgs {
    char* dense[2];             // k, v
    int64_t dense_stride[2];    // bytes between tokens
    char* pool[2];
    const int64_t* slots;
    int64_t T;
    int64_t num_pages;
    int64_t page_stride;
    int64_t row_stride;         // of one head's rows inside a page
    int64_t head_stride;        // 0 in NHD blocks, whose rows are one run
    int64_t s_base;             // KVX_FP4: the same of the scales, from s_base on
    int64_t s_row;
    int64_t s_head;
    int32_t page_size;
    int32_t page_shift;         // log2(page_size), or -1
    uint32_t V;                 // pieces of a row
    uint32_t v_magic;           // ceil(2^32 / V) (0 for V = 1)
    uint32_t VH;                // pieces of a run
    uint32_t vh_magic;
    uint32_t tokens;            // whole rows of a workgroup, or 1 where its threads are fewer than V
    float scale[2];
    float inverse[2];           // 1 / scale, rounded
    unsigned long long* skipped;
};

// A thread's piece x of a token's rows; false: it has none.  Workgroups take
// whole tokens where they can, so that no thread divides by a row's pieces in 64
// bits, and a thread takes its piece of K and of V: one slot, and two rows' loads
// under way (numbered row by row, one piece a thread: reading 49152 tokens 94.7
// us, appending them 69.8).
struct PieceAt {
    int64_t t;
    uint32_t x;
};

__device__ inline bool piece_at(const DenseArgs& A, PieceAt* p) {
    const uint32_t rr = divide(threadIdx.x, A.v_magic);
    p->x = threadIdx.x - rr * A.V + blockIdx.y * blockDim.x;
    p->t = static_cast<int64_t>(blockIdx.x) * A.tokens + rr;
    return rr < A.tokens && p->x < A.V && p->t < A.T;
}

// Where the rows of token t lie in a plane, and of head-major ones the head of
// piece x; false (counted once a token) where the slot is outside the pool.
struct RowAt {
    int64_t page;               // byte offset of the page
    int64_t row;                // row of the page
    uint32_t h;                 // run of the piece
    uint32_t x;                 // piece of the run
};

__device__ inline bool row_at(const DenseArgs& A, const PieceAt& p, RowAt* r) {
    const int64_t slot = A.slots[p.t];
    const int64_t page = A.page_shift >= 0 ? slot >> A.page_shift : slot / A.page_size;
    if (slot < 0 || page >= A.num_pages) {
        if (p.x == 0 && A.skipped != nullptr) atomicAdd(A.skipped, 1ull);
        return false;
    }
    r->page = page * A.page_stride;
    r->row = slot - page * A.page_size;
    r->h = divide(p.x, A.vh_magic);
    r->x = p.x - r->h * A.VH;
    return true;
}

// The numbers' piece (of N bytes) and the block's scale.
template <int N>
__device__ inline int64_t piece_offset(const DenseArgs& A, const RowAt& r) {
    return r.page + r.row * A.row_stride + r.h * A.head_stride + static_cast<int64_t>(r.x) * N;
}
__device__ inline int64_t scale_offset(const DenseArgs& A, const RowAt& r, uint32_t block) {
    return r.page + A.s_base + r.row * A.s_row + r.h * A.s_head + block;
}

// ---------------------------------------------------- writing in 4 bits --
//
// Four neighbouring lanes hold a block, 8 values each, and agree on its largest
// magnitude (a NaN is larger than any as bits); each writes 4 bytes of numbers,
// and the first of a block its scale (joined to words of four scales, by moves
// between lanes, 65536 tokens took the same 70 us).

// Largest of the four lanes of a quad.
__device__ inline uint32_t quad_max(uint32_t x) {
    uint32_t y = __builtin_amdgcn_mov_dpp(x, 0xb1, 0xf, 0xf, true);     // lanes 1 0 3 2
    x = x > y ? x : y;
    y = __builtin_amdgcn_mov_dpp(x, 0x4e, 0xf, 0xf, true);              // lanes 2 3 0 1
    return x > y ? x : y;
}

// The scale byte of a block whose largest magnitude has these bits: the
// exponent of max / 7 rounded up to a power of two.  7 = 1.75 * 2^2, so the
// exponent less 2, and one more where the fraction passes 1.75.
__device__ inline uint32_t block_scale(uint32_t top) {
    if (top > 0x7f800000u) return kNanBlock;
    const int32_t s = static_cast<int32_t>((top + 0x1fffffu) >> 23) - 2;
    return s < static_cast<int32_t>(kLeastBlock) ? kLeastBlock
                                                 : (s > static_cast<int32_t>(kMostBlock) ? kMostBlock : s);
}

template <int FROM>
__device__ inline void widen8(const u32x4 (&x)[2], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (FROM == kFromF32) {
            const uint32_t w = x[i / 4][i % 4];
            f[i] = __builtin_bit_cast(float, w);
        } else {
            const uint32_t w = x[0][i / 2];
            const uint16_t h = static_cast<uint16_t>(i & 1 ? w >> 16 : w);
            if constexpr (FROM == kFromBf16)
                f[i] = __builtin_bit_cast(float, static_cast<uint32_t>(h) << 16);
            else
                f[i] = static_cast<float>(__builtin_bit_cast(_Float16, h));
        }
    }
}

template <int FROM, bool SCALED, bool PAST>
__global__ __launch_bounds__(kAppendThreads) void k_append_fp4(const DenseArgs A) {
    PieceAt p;
    if (!piece_at(A, &p)) return;
    constexpr int N = FROM == kFromF32 ? 2 : 1;
    u32x4 x[2][2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const char* s = A.dense[kv] + p.t * A.dense_stride[kv] + static_cast<int64_t>(p.x) * (16 * N);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const u32x4* y = reinterpret_cast<const u32x4*>(s) + j;
            x[kv][j] = PAST ? __builtin_nontemporal_load(y) : *y;
        }
    }
    RowAt r;
    if (!row_at(A, p, &r)) return;                      // the same for a row's lanes
    const int64_t at = piece_offset<4>(A, r), scale_at = scale_offset(A, r, r.x / 4);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        float f[8];
        widen8<FROM>(x[kv], f);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the quotient's remainder loses the sign of a zero
            if constexpr (SCALED)
                f[i] = __builtin_copysignf(quotient(f[i], A.scale[kv], A.inverse[kv]), f[i]);
            const uint32_t b = __builtin_bit_cast(uint32_t, f[i]) & 0x7fffffffu;
            top = top > b ? top : b;
        }
        const uint32_t byte = block_scale(quad_max(top));
        const float unit = __builtin_bit_cast(float, byte << 23);
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], unit, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], unit, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], unit, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], unit, 3);
        if (byte == kNanBlock) w = 0;
        *reinterpret_cast<uint32_t*>(A.pool[kv] + at) = w;
        if ((threadIdx.x & 3) == 0)
            *reinterpret_cast<uint8_t*>(A.pool[kv] + scale_at) = static_cast<uint8_t>(byte);
    }
}

// ------------------------------------------------------------- reading --
//
// Row t of k and of v is the row of slot slots[t]: the same bytes, or e4m3 or
// 4-bit values times scale in the dense rows' type (one rounding, of the 32-bit
// product).  A thread takes 8 values, or 16 bytes where they are copied.

enum : int { kReadBytes = 0, kReadFp8 = 1, kReadFp4 = 2 };

template <bool PAST>
__device__ inline void store16(char* to, u32x4 w) {
    u32x4* y = reinterpret_cast<u32x4*>(to);
    if constexpr (PAST)
        __builtin_nontemporal_store(w, y);
    else
        *y = w;
}

template <int TO, bool PAST>
__device__ inline void store8(char* to, const float (&f)[8]) {
    if constexpr (TO == kFromF32) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, f[4 * j + i]);
            store16<PAST>(to + 16 * j, w);
        }
    } else {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TO == kFromBf16) {
                const bf16x2 y = {static_cast<__bf16>(f[2 * i]), static_cast<__bf16>(f[2 * i + 1])};
                w[i] = __builtin_bit_cast(uint32_t, y);
            } else {
                const f16x2 y = {static_cast<_Float16>(f[2 * i]), static_cast<_Float16>(f[2 * i + 1])};
                w[i] = __builtin_bit_cast(uint32_t, y);
            }
        }
        store16<PAST>(to, w);
    }
}

// HOW: how the pool holds the values; TO: kFromBf16, kFromF16 or kFromF32, the
// dense rows' type (any where bytes are copied).
template <int HOW, int TO, bool PAST>
__global__ __launch_bounds__(kAppendThreads) void k_read(const DenseArgs A) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    PieceAt p;
    RowAt r;
    if (!piece_at(A, &p) || !row_at(A, p, &r)) return;
    constexpr int N = HOW == kReadBytes ? 16 : (TO == kFromF32 ? 32 : 16);
    constexpr int IN = HOW == kReadBytes ? 16 : (HOW == kReadFp8 ? 8 : 4);
    const int64_t at = piece_offset<IN>(A, r);
    uint32_t w[2][IN / 4], byte[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const char* from = A.pool[kv] + at;
        if constexpr (IN == 16) {
            const u32x4 y = *reinterpret_cast<const u32x4*>(from);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[kv][i] = y[i];
        } else if constexpr (IN == 8) {
            const u32x2 y = *reinterpret_cast<const u32x2*>(from);
            w[kv][0] = y.x;
            w[kv][1] = y.y;
        } else {
            w[kv][0] = *reinterpret_cast<const uint32_t*>(from);
            byte[kv] = *reinterpret_cast<const uint8_t*>(A.pool[kv] + scale_offset(A, r, r.x / 4));
        }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        char* to = A.dense[kv] + p.t * A.dense_stride[kv] + static_cast<int64_t>(p.x) * N;
        if constexpr (HOW == kReadBytes) {
            store16<PAST>(to, u32x4{w[kv][0], w[kv][1], w[kv][2], w[kv][3]});
        } else {
            float f[8];
            auto pair = [&](int i, f32x2 y) {
                f[2 * i] = y.x * A.scale[kv];
                f[2 * i + 1] = y.y * A.scale[kv];
            };
            if constexpr (HOW == kReadFp8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    pair(2 * i, __builtin_amdgcn_cvt_pk_f32_fp8(w[kv][i], false));
                    pair(2 * i + 1, __builtin_amdgcn_cvt_pk_f32_fp8(w[kv][i], true));
                }
            } else {
                // the conversion takes the exponent's bits: 0 is 2^-127, and 255 makes NaN
                const float unit = __builtin_bit_cast(float, byte[kv] << 23);
                pair(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][0], unit, 0));
                pair(1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][0], unit, 1));
                pair(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][0], unit, 2));
                pair(3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][0], unit, 3));
            }
            store8<TO, PAST>(to, f);
        }
    }
}

}  // namespace tables
}  // namespace kvx
