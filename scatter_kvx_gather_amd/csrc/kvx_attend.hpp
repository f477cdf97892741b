// kvx_attend.hpp -- attention over a paged pool for batches whose requests
// share prefixes (gfx950 / CDNA4).
//
// Mathematics.  Query token i of request r (n tokens, context c) sees every
// key of its group's prefix and, in its own context, keys 0 .. c - n + i
// (all c of them without the causal flag).  With s = scale * q.k,
//   m = max s,  l = sum 2^(s' - m'),  o = sum 2^(s' - m') v   (s' = s log2 e)
// over any subset of the keys, and two subsets join by
//   m = max(m1, m2),  l = l1 2^(m1-m) + l2 2^(m2-m),  o likewise,
// so a prefix is computed once for all rows of its group, a long axis is cut
// anywhere, and out = o / l, lse = m + ln l at the end.  m, l and o are 32
// bits throughout; weights are rounded to the query's type for the second
// product (relative 2^-8 at most for bf16, 2^-11 for f16, averaged over the
// keys), while l sums them unrounded.
//
// Work.  A segment is a group's prefix or a request's own context; an item is
// (segment, head set, tile of query rows), and its length is the number of
// keys its last row sees, and some units more that stand for its fixed time.
// All items laid end to end make one line that the workgroups cut into equal
// pieces, whatever the lengths are: they
// stand in device memory, so each workgroup finds its piece itself from a
// scan over the segments, and the host needs to know none of them.  A piece
// that is not a whole item leaves (m, l, o) in the workgroup's two slots of
// the workspace; a whole item of a row that has two parts (prefix and own)
// leaves them in that part's row buffer; a whole item of a row with one part
// is written out at once.  k_attend_join joins the rest.
//
// Thin tiles (16 query rows a wave) are for segments with few rows, where the
// KV rows' bytes are the bound: the waves of a workgroup take the heads of
// one key range, so a pool row is read whole by one workgroup, and K and V go
// from memory to the matrix instructions through registers alone, a step of 32
// keys ahead, page ids two.  256 requests behind 256 to 2048 tokens, 8 kv heads
// of 128 dims: 255 us, 4.9 TB/s (a copy of 2 GiB: 4.91, read and written).
//
// Wide tiles (128 or 256 rows a workgroup) are for segments with many rows,
// where the matrix units and what feeds them are the bound: 64 or 128 keys at a
// time go from memory to one of two buffers in shared memory without passing
// registers, and each wave reads them for its 32 rows (16 above 128 dims).
// 8 prompts of 2048 tokens, 32 heads over 8 of 128 dims: 397 us, 693 TFLOP/s;
// with 64 dims 2 prompts of 8192 740 TFLOP/s, with 256 2 of 4096 615.  Of a
// tile's 10 thousand cycles the products' own are 4.1; the exponentials and
// their packing come next, then loads issued and waits at the end of a tile.
// Two steps of 32 keys together, their products in the shadow of each other's
// softmax, and half of the waves staging after their first step beat one step
// (664 -> 442 us with the split items' join, 410 -> 397).
//
// The second launch joins what is split: 3 to 10 us where that is a chain of its
// launch and three dependent loads, more where its bytes count: behind a prefix
// every row has two parts, of which it reads 32-bit partial rows (256 requests
// of 64 heads 15 us, 8 chunks of 100 to 256 tokens of 32 heads, 47 MB, 26 us).
//
// Fragments.  S^T = K Q^T by 16x16x32 products: K rows are loaded as the A
// operand holds them (lane a + 16 g: key a, 8 dims at 8 g).  The result has
// query row a in lanes a + 16 g, keys 4 g + r of two 16-key tiles, which is
// how the B operand of O^T = V^T P^T holds them when its 8 k-slots of lane
// group g stand for keys {4g..4g+3, 16+4g..16+4g+3}: the weights never leave
// their registers.  V's operand is a transposition of its rows.  Thin tiles
// load V row by row (lane a: dims 8a .. 8a+7 of the group's 8 keys) and
// transpose 8 x 8 blocks in registers with byte permutes; row a of the j-th
// product is then dim 8 a + j.  Wide tiles read rows from shared memory with
// transposing reads; row a of the j-th product is dim 16 j + a.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace kvx {
namespace attend {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8;               // waves of an attention workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kKeys = 32;               // keys of one step of a wave
constexpr int kThinRows = 16;
constexpr int32_t kMaxKeys = 1 << 30;    // of a context or a prefix: step indices stay in 32 bits
constexpr int kJoinWaves = 8;
constexpr int kJoinParts = 4;

// Weights are taken against a reference, which is a row's maximum less kRoom
// when it moves and may lag it while a lane's weights of one step sum to no
// more than kMostWeight.  f16's weights start at 2^8, or those below 2^-14 of
// the largest would be subnormal and, where many are alike, rounded to one
// side together; so they have eight bits more, and stay below f16's largest.
template <class T>
constexpr float kRoom = std::is_same_v<T, _Float16> ? 8.0f : 0.0f;
template <class T>
constexpr float kMostWeight = std::is_same_v<T, _Float16> ? 32768.0f : 256.0f;
// The reference of a row that has seen no key: any score's weight against it
// is infinite, and -inf's is 0.
constexpr float kNoKey = -3.0e38f;

// The lane, as a value that the compiler does not carry around loops: what is
// computed from it stays where it is used.  Held over the loops of a piece,
// lane-dependent addresses and predicates of every path filled the registers
// and the loops' own values went to scratch memory.
__device__ inline int here_lane() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// The item that reaches from a workgroup's piece into a later one's, if there is one.
struct Split {
    int64_t item;                       // its first unit
    int32_t last;                       // the piece that it ends in; -1: no such item
    int32_t w, slot0;                   // the piece that it begins in, the line's first slot
    int32_t wide;
    int32_t tok0, ntok;                 // of its segment
    int32_t set, tile;
    int32_t keys;                       // that its last row sees
    int32_t extra;
    int32_t pad[2];
};

struct Lists {                          // where a kind of segment's keys live
    const int64_t* pg_off;
    const int32_t* ids;
    int64_t num_ids;
};

struct Args {
    const char* k;                      // the layer's planes
    const char* v;
    int64_t row_stride;                 // bytes between the rows of a page, of one head
    int64_t page_stride;
    int64_t head_stride;
    int64_t num_pages;
    int32_t page_size;
    int32_t page_shift;                 // log2(page_size), or -1
    const int64_t* tok_off;             // [num_reqs + 1]
    const int32_t* ctx;                 // [num_reqs]
    const int64_t* grp_off;             // [num_groups + 1]
    const int32_t* plen;                // [num_groups]
    Lists own;
    Lists pre;
    const char* q;
    char* out;
    float* lse;                         // or NULL
    int64_t q_stride;                   // bytes between tokens
    int64_t out_stride;
    unsigned long long* skipped;        // or NULL
    int32_t T;                          // query tokens
    int32_t num_reqs;
    int32_t num_groups;
    int32_t H;                          // kv heads
    int32_t G;                          // query heads per kv head
    int32_t D;
    int32_t causal;
    float scale;                        // softmax scale * k scale * log2 e
    float v_scale;
    // tilings: thin heads are (kv head, part of its query heads) pairs
    int32_t parts;                      // parts of a kv head's query heads
    int32_t gv;                         // query heads of a part (the last may have fewer)
    int32_t sets;                       // head sets of a thin segment
    int32_t hs;                         // thin heads per set
    int32_t kp;                         // waves that share a thin head's keys
    int32_t thin_tokens;                // tokens per thin tile
    int32_t wide_tokens;                // tokens per wide tile
    int32_t pre_wide;                   // prefixes run in wide tiles
    int32_t own_wide;                   // own contexts run in wide tiles
    int32_t thin_min_log2;              // fewest units of a piece
    int32_t wide_min_log2;
    int32_t thin_item;                  // units that an item's fixed time counts for
    int32_t wide_item;
    float wide_weight;                  // time of a wide key over a thin key's
    // workspace
    struct Placed* placed;              // [num_groups + num_reqs]: segments on their lines
    int64_t* plan;                      // [6]: Cuts of the thin and the wide line, workgroups of each
    struct Split* splits;               // [grid], by slot / 2
    float* slot_o;                      // [2 * grid][slot rows][D]
    float* slot_ml;                     // [2 * grid][slot rows][2]
    float* row_o;                       // [2][T][Hq][D]: own, prefix (only with prefixes)
    float* row_ml;                      // [2][T][Hq][2]
    int32_t slot_rows;
};

// A value that is the same in every lane, in a scalar register: what is loaded
// from memory that the kernel might write comes in vector registers otherwise,
// and so does all that is computed from it.
__device__ inline int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ inline int64_t uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
    return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// ------------------------------------------------------------- segments --

struct Seg {
    int32_t tok0;                       // first query token
    int32_t ntok;
    int32_t keys;
    int32_t base;                       // keys the token before the first would see
    int32_t tiles;
    int32_t tp;                         // tokens per tile
    int32_t sets;                       // head sets
    int32_t extra;                      // units of a tile's fixed time
    bool wide;
    bool causal;
};

__device__ inline int32_t clamp_to(int64_t x, int64_t lo, int64_t hi) {
    return static_cast<int32_t>(x < lo ? lo : (x > hi ? hi : x));
}

// Segment s: prefix s of group s, or the own context of request s - groups.
// (Offsets that break their contract are held inside the batch.)
__device__ inline Seg segment(const Args& A, int32_t s) {
    Seg g;
    const bool pre = s < A.num_groups;
    int32_t r0 = s - A.num_groups, r1 = r0 + 1, keys;
    if (pre) {
        r0 = clamp_to(A.grp_off[s], 0, A.num_reqs);
        r1 = clamp_to(A.grp_off[s + 1], r0, A.num_reqs);
        keys = A.plen[s];
    } else {
        keys = A.ctx[r0];
    }
    g.keys = clamp_to(keys, 0, kMaxKeys);
    g.tok0 = clamp_to(A.tok_off[r0], 0, A.T);
    g.ntok = clamp_to(A.tok_off[r1], g.tok0, A.T) - g.tok0;
    g.causal = !pre && A.causal != 0;
    g.base = !g.causal ? g.keys : (g.keys > g.ntok ? g.keys - g.ntok : 0);
    g.wide = (pre ? A.pre_wide : A.own_wide) != 0;
    g.tp = g.wide ? A.wide_tokens : A.thin_tokens;
    g.sets = g.wide ? A.H : A.sets;
    g.extra = g.wide ? A.wide_item : A.thin_item;
    g.tiles = g.keys > 0 ? (g.ntok + g.tp - 1) / g.tp : 0;
    return g;
}

__device__ inline Seg uniform(const Seg& g) {
    Seg u;
    u.tok0 = uniform(g.tok0);
    u.ntok = uniform(g.ntok);
    u.keys = uniform(g.keys);
    u.base = uniform(g.base);
    u.tiles = uniform(g.tiles);
    u.tp = uniform(g.tp);
    u.sets = uniform(g.sets);
    u.extra = uniform(g.extra);
    u.wide = uniform(static_cast<int32_t>(g.wide)) != 0;
    u.causal = uniform(static_cast<int32_t>(g.causal)) != 0;
    return u;
}

// Units before tile i of a head set, the keys of tile i (one more row tile of a
// causal segment sees up to tp more keys), and the units of a head set.
__device__ inline int64_t tile_start(const Seg& g, int32_t i) {
    const int64_t n = i;
    return n * (static_cast<int64_t>(g.base) + g.extra) + (g.causal ? g.tp * (n * (n + 1) / 2) : 0);
}
__device__ inline int64_t tile_keys(const Seg& g, int32_t i) {
    if (!g.causal) return g.base;
    const int64_t last = (static_cast<int64_t>(i) + 1) * g.tp;
    return g.base + (last < g.ntok ? last : g.ntok);
}
__device__ inline int64_t set_units(const Seg& g) {
    return g.tiles > 0 ? tile_start(g, g.tiles - 1) + tile_keys(g, g.tiles - 1) + g.extra : 0;
}
// The key that a cut x units into an item falls on: a whole step of 2^log2 keys,
// or the item's end (`keys`: an item is longer than its segment has keys where a
// causal segment has more tokens than keys).
__device__ inline int32_t cut_key(const Seg& g, int64_t x, int step_log2, int32_t keys) {
    if (x <= g.extra) return 0;
    const int64_t k = (x - g.extra) >> step_log2 << step_log2;
    return k < keys ? static_cast<int32_t>(k) : keys;
}

// A line of n units cut into `wgs` pieces whose lengths differ by one at most.
struct Cuts {
    int64_t q, r;               // r pieces of q + 1 units, then pieces of q
    __device__ inline Cuts() {}
    __device__ inline Cuts(int64_t n, int64_t wgs) {
        q = wgs > 0 ? n / wgs : 0;
        r = n - q * wgs;
    }
    __device__ inline int64_t start(int64_t w) const { return q * w + (w < r ? w : r); }
    __device__ inline int64_t piece_of(int64_t x) const {
        const int64_t big = (q + 1) * r;
        return x < big ? x / (q + 1) : r + (x - big) / q;
    }
};

// A segment as k_attend leaves it for the join.
struct Placed {
    Seg g;
    int64_t start;              // its first unit on its line
    int64_t units;              // of a head set
};

// Page id of key t (any id when the list has no such entry), and the byte
// offset of the key's row (of head 0) from it, or -1 when entry or page are out
// of range.  Two steps, because loops load the ids of a later step first and
// ask for the offsets a step later: loads return in order, so an id asked for
// at once would wait for the rows under way before it.  The load has no
// condition, which would do the same.
__device__ inline int32_t key_page(const Args& A, const Lists& L, int64_t pg0, int32_t t) {
    const uint32_t tu = static_cast<uint32_t>(t);
    const int64_t kp = A.page_shift >= 0 ? tu >> A.page_shift : tu / static_cast<uint32_t>(A.page_size);
    int64_t i = 0;
    if (pg0 >= -kp && pg0 < L.num_ids - kp) i = pg0 + kp;
    // an empty list's entry is read from an array that is never empty
    const int32_t* ids = L.num_ids > 0 ? L.ids : reinterpret_cast<const int32_t*>(A.tok_off);
    return ids[i];
}
__device__ inline int64_t page_offset(const Args& A, const Lists& L, int64_t pg0, int32_t page,
                                      int32_t t, int32_t end) {
    const uint32_t tu = static_cast<uint32_t>(t), b = static_cast<uint32_t>(A.page_size);
    const int64_t kp = A.page_shift >= 0 ? tu >> A.page_shift : tu / b;
    const uint32_t row = A.page_shift >= 0 ? tu & (b - 1) : tu - static_cast<uint32_t>(kp) * b;
    // the index is range-checked before the sum is formed: no pg_off value makes it wrap
    const bool ok = (t < end) & (pg0 >= -kp) & (pg0 < L.num_ids - kp) & (page >= 0) &
                    (page < A.num_pages);
    const int64_t off = static_cast<uint32_t>(page) * A.page_stride + row * A.row_stride;
    return ok ? off : -1;
}
__device__ inline int64_t key_offset(const Args& A, const Lists& L, int64_t pg0, int32_t t,
                                     int32_t end) {
    return page_offset(A, L, pg0, key_page(A, L, pg0, t), t, end);
}

// ------------------------------------------------------------ elements --

template <class T>
struct Mma;
template <>
struct Mma<__bf16> {
    static __device__ f32x4 run(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ uint32_t pack(float x, float y) {
        bf16x2 r = {static_cast<__bf16>(x), static_cast<__bf16>(y)};
        return __builtin_bit_cast(uint32_t, r);
    }
    template <bool HI>
    static __device__ uint32_t from_fp8(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
    }
    static __device__ float lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
    static __device__ float hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }
    static constexpr uint32_t kExp = 0x7f807f80u;       // exponent bits of both halves
};
template <>
struct Mma<_Float16> {
    static __device__ f32x4 run(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    static __device__ uint32_t pack(float x, float y) {
        f16x2 r = {static_cast<_Float16>(x), static_cast<_Float16>(y)};
        return __builtin_bit_cast(uint32_t, r);
    }
    template <bool HI>
    static __device__ uint32_t from_fp8(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
    }
    static __device__ float lo(uint32_t w) {
        return static_cast<float>(__builtin_bit_cast(f16x2, w).x);
    }
    static __device__ float hi(uint32_t w) {
        return static_cast<float>(__builtin_bit_cast(f16x2, w).y);
    }
    static constexpr uint32_t kExp = 0x7c007c00u;
};

// w with 16-bit halves that are an infinity or a NaN cleared; of a word of four
// fp8 values, with NaN cleared.
template <class T>
__device__ inline uint32_t finite_pair(uint32_t w) {
    constexpr uint32_t lo = Mma<T>::kExp & 0xffffu, hi = Mma<T>::kExp & 0xffff0000u;
    return ((w & lo) == lo ? 0u : w & 0xffffu) | ((w & hi) == hi ? 0u : w & 0xffff0000u);
}
__device__ inline uint32_t finite_quad(uint32_t w) {
    const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    return w & ~((nan >> 7) * 0xffu);
}

// Shapes of one (query type, pool element, padded head dim) combination.
template <class T, bool FP8, int DP>
struct Cfg {
    static constexpr int EB = FP8 ? 1 : 2;
    static constexpr int KS = DP / 32;                  // k-steps of the first product
    static constexpr int NK = DP * EB / 64;             // 16-byte loads of K per key tile
    static constexpr int VE = DP >= 128 ? 8 : 4;        // dims of V a lane holds per chunk
    static constexpr int NC = DP / (16 * VE);           // chunks of V
    static constexpr int VW = VE * EB / 4;              // dwords of a V chunk as loaded
    static constexpr int NJ = NC * VE;                  // products of the second product
};

// First dim of the 8 that k-step ks takes from lane group g.
template <class C>
__device__ inline int k_dim(int ks, int g) {
    return C::EB == 2 ? ks * 32 + g * 8 : (ks >> 1) * 64 + g * 16 + (ks & 1) * 8;
}

template <int W>
struct Words {
    uint32_t w[W];
};

template <int W>
__device__ inline Words<W> load_words(const char* p) {
    Words<W> r;
    if constexpr (W == 4) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(p);
        r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
    } else if constexpr (W == 2) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(p);
        r.w[0] = x.x; r.w[1] = x.y;
    } else {
        r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
    return r;
}

// K of one 16-key tile as loaded, and its k-step ks as the product takes it.
template <class C>
struct KTile {
    u32x4 raw[C::NK];
};

template <class C>
__device__ inline void load_k(KTile<C>* t, const char* row, int g, int D) {
#pragma unroll
    for (int x = 0; x < C::NK; ++x) {
        const int b = x * 64 + g * 16;
        const bool in = b < D * C::EB;
        t->raw[x] = *reinterpret_cast<const u32x4*>(row + (in ? b : 0));
    }
}

template <class T, class C>
__device__ inline u32x4 k_frag(const KTile<C>& t, int ks, int g, int D) {
    u32x4 f;
    if constexpr (C::EB == 2) {
        f = t.raw[ks];
    } else {
        const u32x4 r = t.raw[ks >> 1];
        const uint32_t lo = (ks & 1) ? r.z : r.x, hi = (ks & 1) ? r.w : r.y;
        f = u32x4{Mma<T>::template from_fp8<false>(lo), Mma<T>::template from_fp8<true>(lo),
                  Mma<T>::template from_fp8<false>(hi), Mma<T>::template from_fp8<true>(hi)};
    }
    // dims past the head: another head's values must not meet the query's zeros
    // (an infinity there would make a NaN)
    if (D < C::KS * 32 && k_dim<C>(ks, g) >= D) f = u32x4{0, 0, 0, 0};
    return f;
}

// V of the 8 keys of a lane group, one chunk, in the query's type: x[i][w] = dims 2w, 2w+1 of key i.
template <class T, class C>
__device__ inline void v_pairs(const Words<C::VW>& raw, uint32_t* x) {
    if constexpr (C::EB == 2) {
#pragma unroll
        for (int w = 0; w < C::VE / 2; ++w) x[w] = raw.w[w];
    } else {
#pragma unroll
        for (int w = 0; w < C::VW; ++w) {
            x[2 * w] = Mma<T>::template from_fp8<false>(raw.w[w]);
            x[2 * w + 1] = Mma<T>::template from_fp8<true>(raw.w[w]);
        }
    }
}

// Operands of dims 2w and 2w+1 from the pairs of 8 keys.
__device__ inline void v_transpose(const uint32_t (&x)[8], u32x4* even, u32x4* odd) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        (*even)[p] = __builtin_amdgcn_perm(x[2 * p + 1], x[2 * p], 0x05040100u);
        (*odd)[p] = __builtin_amdgcn_perm(x[2 * p + 1], x[2 * p], 0x07060302u);
    }
}

// ------------------------------------------------------ running softmax --

// State of 16 query rows: the lane's row a = lane % 16.
template <class C>
struct Rows {
    float m;                    // reference maximum (log2), the same in a row's four lanes
    float ref;                  // m, or kNoKey while it is -inf
    float l;                    // this lane's share of the sum
    f32x4 o[C::NJ];             // thin o[c * VE + j][r]: dim 16 VE c + (4 g + r) VE + j
                                // wide o[j][r]: dim 16 j + 4 g + r
};

template <class C>
__device__ inline void clear(Rows<C>* R) {
    R->m = -INFINITY;
    R->ref = kNoKey;
    R->l = 0.0f;
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) R->o[j] = f32x4{0, 0, 0, 0};
}

// Scores s of 32 U keys to weights in the query's type.  The weights are taken
// against the row's reference maximum as it stands, and only when a lane's sum
// of them passes kMostWeight (or is a NaN) is the maximum looked for, the
// accumulators rescaled and the weights taken anew: looking for it every time
// cost as many instructions as the rest.
template <class T, class C, int U>
__device__ inline float take_weights(const Rows<C>& R, const f32x4* s, float scale, u32x4* pf) {
    float part[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * u + (i >> 2)][i & 3], scale, -R.ref));
            part[i & 1] += p[i];
        }
        pf[u] = u32x4{Mma<T>::pack(p[0], p[1]), Mma<T>::pack(p[2], p[3]), Mma<T>::pack(p[4], p[5]),
                      Mma<T>::pack(p[6], p[7])};
    }
    return part[0] + part[1];
}

template <class T>
__device__ inline bool too_much(float sum) {
    return __any(!(sum <= kMostWeight<T>));
}

template <class T, class C, int U>
__device__ inline float move_maximum(Rows<C>* R, const f32x4* s, float scale, u32x4* pf) {
    float top = -INFINITY;
#pragma unroll
    for (int x = 0; x < 2 * U; ++x)
        top = fmaxf(fmaxf(fmaxf(top, s[x][0]), s[x][1]), fmaxf(s[x][2], s[x][3]));
    top *= scale;
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m = fmaxf(R->m, top - kRoom<T>);
    const float a = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(R->m - m);
    R->m = m;
    R->ref = m == -INFINITY ? kNoKey : m;
    R->l *= a;
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) R->o[j] *= a;
    return take_weights<T, C, U>(*R, s, scale, pf);
}

// In a matrix product a weight of 0 times an infinity or a NaN is a NaN, so in
// steps in which some row does not see some key, values that are not finite
// are left out of the product.  What they make of the rows that do see them,
// whose weights are positive, is added here: the value itself.  Rare, and a V
// row at a time from memory.  Keys [from, to); `limit` is the lane's row's.
template <class T, class C, bool WIDE>
__device__ inline void add_not_finite(const Args& A, const Lists& L, int64_t pg0, const char* vhead,
                                      int32_t from, int32_t to, int32_t limit, Rows<C>* R) {
    const int g = here_lane() >> 4;
#pragma unroll 1
    for (int32_t t = from; t < to; ++t) {
        const int64_t off = key_offset(A, L, pg0, t, to);
        if (off < 0) continue;
#pragma unroll
        for (int x = 0; x < C::NJ; ++x) {
            // four dims in a run, as store_rows has them
            constexpr int Q = C::VE / 4;
            const int c = x / (4 * Q), r = x / Q % 4, j = c * C::VE + x % Q * 4;
            const int d = WIDE ? x * 16 + 4 * g : c * 16 * C::VE + (4 * g + r) * C::VE + x % Q * 4;
            if (d >= A.D || t >= limit) continue;
            uint32_t w[2];
            if constexpr (C::EB == 2) {
                const u32x2 y = *reinterpret_cast<const u32x2*>(vhead + off + d * 2);
                w[0] = y.x;
                w[1] = y.y;
            } else {
                const uint32_t y = *reinterpret_cast<const uint32_t*>(vhead + off + d);
                w[0] = Mma<T>::template from_fp8<false>(y);
                w[1] = Mma<T>::template from_fp8<true>(y);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = i & 1 ? Mma<T>::hi(w[i >> 1]) : Mma<T>::lo(w[i >> 1]);
                float* o = WIDE ? &reinterpret_cast<float*>(&R->o[x])[i]
                                : &reinterpret_cast<float*>(&R->o[j + i])[r];
                if (!__builtin_isfinite(v)) *o += v;
            }
        }
    }
}

// ------------------------------------------------------------- results --

enum : int { kSlot = 0, kRowBuffer = 1, kFinal = 2 };

// Where a piece's rows go.
struct Dest {
    int kind;
    int32_t slot;               // kSlot
    int part;                   // kRowBuffer: 0 own, 1 prefix
};

template <class T, class C, bool WIDE>
__device__ inline void store_rows(const Args& A, const Dest& to, const Rows<C>& R, int slot_row,
                                  int32_t token, int32_t head, bool live) {
    const int lane = here_lane(), g = lane >> 4;
    float l = R.l;
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (!live) return;
    // runs of 4 dims: f(dim, values)
    auto each = [&](auto f) {
#pragma unroll
        for (int x = 0; x < C::NJ; ++x) {
            if constexpr (WIDE) {
                f(x * 16 + 4 * g, R.o[x]);
            } else {
                constexpr int Q = C::VE / 4;                // runs of a row r of a chunk
                const int c = x / (4 * Q), r = x / Q % 4, j = c * C::VE + x % Q * 4;
                f(c * 16 * C::VE + (4 * g + r) * C::VE + x % Q * 4,
                  f32x4{R.o[j][r], R.o[j + 1][r], R.o[j + 2][r], R.o[j + 3][r]});
            }
        }
    };
    const int64_t out_row = static_cast<int64_t>(token) * A.H * A.G + head;
    if (to.kind == kFinal) {
        const float inv = l == 0.0f ? 0.0f : A.v_scale / l;
        char* row = A.out + static_cast<int64_t>(token) * A.out_stride + static_cast<int64_t>(head) * A.D * 2;
        each([&](int d, const f32x4& x) {
            if (d < A.D)
                *reinterpret_cast<u32x2*>(row + d * 2) =
                    u32x2{Mma<T>::pack(x[0] * inv, x[1] * inv), Mma<T>::pack(x[2] * inv, x[3] * inv)};
        });
        if (g == 0 && A.lse != nullptr)
            A.lse[out_row] =
                l == 0.0f ? -INFINITY : (R.m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
        return;
    }
    float *o, *ml;
    if (to.kind == kSlot) {
        const int64_t row = static_cast<int64_t>(to.slot) * A.slot_rows + slot_row;
        o = A.slot_o + row * A.D;
        ml = A.slot_ml + row * 2;
    } else {
        const int64_t row = static_cast<int64_t>(to.part) * A.T * A.H * A.G + out_row;
        o = A.row_o + row * A.D;
        ml = A.row_ml + row * 2;
    }
    if (g == 0) *reinterpret_cast<float2*>(ml) = make_float2(R.m, l);
    each([&](int d, const f32x4& x) {
        if (d < A.D) *reinterpret_cast<f32x4*>(o + d) = x;
    });
}

// --------------------------------------------------------------- thin --

// A piece of an item: keys [key0, key1) of tile `tile` of head set `set`.
struct Piece {
    Seg seg;
    Lists lists;
    int64_t pg0;
    int32_t set;
    int32_t tile;
    int32_t key0, key1;
    bool counts;                // this piece counts the out-of-range keys
};

// Counts the out-of-range keys of a piece's range, once per key of a segment:
// the pieces of the segment's last tile (which sees every key) and first head
// set cover its keys exactly once.
__device__ inline void count_skipped(const Args& A, const Piece& P, int wave) {
    if (A.skipped == nullptr || !P.counts) return;
    const int lane = threadIdx.x & 63;
    unsigned long long n = 0;
    for (int64_t t = static_cast<int64_t>(P.key0) + wave * 64; t < P.key1; t += kThreads) {
        const int32_t k = static_cast<int32_t>(t) + lane;
        const bool bad = k < P.key1 && key_offset(A, P.lists, P.pg0, k, P.key1) < 0;
        n += __popcll(__ballot(bad));
    }
    if (lane == 0 && n != 0) atomicAdd(A.skipped, n);
}

template <class T, class C>
__device__ inline void load_q(const Args& A, u32x4 (&q)[C::KS], int32_t token, int32_t head,
                              bool live) {
    const int g = here_lane() >> 4;
    const char* row = A.q + static_cast<int64_t>(token) * A.q_stride + static_cast<int64_t>(head) * A.D * 2;
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
        const int d = k_dim<C>(ks, g);
        q[ks] = u32x4{0, 0, 0, 0};
        if (live && d < A.D) q[ks] = *reinterpret_cast<const u32x4*>(row + d * 2);
    }
}

// Keys this lane's row does not see get -inf: key index key0 + ..., seen below
// `limit` and where `valid` has its bit.
__device__ inline void mask_scores(f32x4* s, int32_t key0, int32_t limit, uint32_t valid) {
    const int g = here_lane() >> 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int key = (i >> 2) * 16 + 4 * g + (i & 3);
        const bool seen = (key0 + key < limit) & (((valid >> key) & 1) != 0);
        s[i >> 2][i & 3] = seen ? s[i >> 2][i & 3] : -INFINITY;
    }
}

template <class T, class C>
__device__ void run_thin(const Args& A, const Piece& P, const Dest& to, float* lds) {
    const int lane = here_lane(), a = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = wave % A.hs, part = wave / A.hs;
    const int32_t vh = P.set * A.hs + h;                  // thin head
    const int32_t kvh = vh / A.parts, sub = vh % A.parts;
    const bool works = part < A.kp && vh < A.H * A.parts;
    count_skipped(A, P, wave);

    // this lane's query row
    const int32_t local = P.tile * A.thin_tokens + a / A.gv;
    const int32_t hsub = sub * A.gv + a % A.gv;
    const bool live = works && a < A.thin_tokens * A.gv && local < P.seg.ntok && hsub < A.G;
    const int32_t token = P.seg.tok0 + local;
    const int32_t head = kvh * A.G + hsub;
    const int32_t past = P.seg.keys - P.seg.ntok;
    // keys that this row sees, and the fewest that a row of the tile sees
    int32_t limit = P.key1, all_see = P.key1;
    if (P.seg.causal) {
        if (live && past + local + 1 < limit) limit = past + local + 1;
        all_see = past + P.tile * A.thin_tokens + 1;
    }

    Rows<C> R;
    clear(&R);
    if (works) {
        u32x4 q[C::KS];
        load_q<T, C>(A, q, token, head, live);
        const char* kh = A.k + kvh * A.head_stride;
        const char* vhd = A.v + kvh * A.head_stride;
        const int32_t step = kKeys * A.kp;

        // K and V of a step as loaded.  Up to 128 dims both are loaded a step
        // ahead; above, K and then V of the present step, or they would not
        // fit the registers (64 contexts of 2048 keys 64 us, a step ahead 72).
        constexpr bool AHEAD = C::NC == 1;
        KTile<C> kt[2];
        Words<C::VW> vr[8][C::NC];
        // page ids of a step's keys, one per lane, and their offsets
        auto page_of = [&](int32_t key0) -> int32_t {
            return key_page(A, P.lists, P.pg0, key0 + (lane & 31));
        };
        auto offset_of = [&](int32_t key0, int32_t page) -> int64_t {
            return page_offset(A, P.lists, P.pg0, page, key0 + (lane & 31), P.key1);
        };
        auto load_keys = [&](int64_t off) {
            const int64_t safe = off < 0 ? 0 : off;
#pragma unroll
            for (int x = 0; x < 2; ++x) load_k<C>(&kt[x], kh + __shfl(safe, x * 16 + a), g, A.D);
        };
        auto load_values = [&](int64_t off) {
            const int64_t safe = off < 0 ? 0 : off;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const char* row = vhd + __shfl(safe, (i >> 2) * 16 + 4 * g + (i & 3));
#pragma unroll
                for (int c = 0; c < C::NC; ++c) {
                    const int d = (c * 16 + a) * C::VE;
                    vr[i][c] = load_words<C::VW>(row + (d < A.D ? d * C::EB : 0));
                }
            }
        };
        // operands of products 2 w and 2 w + 1 of chunk c
        auto value_pair = [&](int c, int w, u32x4* even, u32x4* odd) {
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t x[C::VE / 2];
                v_pairs<T, C>(vr[i][c], x);
                y[i] = x[w];
            }
            v_transpose(y, even, odd);
        };

        int32_t first_odd = -1;         // this wave's first step whose product left values out
        int32_t key0 = P.key0 + part * kKeys;
        int32_t page = -1;
        int64_t off = -1;
        if (key0 < P.key1) {
            off = offset_of(key0, page_of(key0));
            page = page_of(key0 + step);
            if (AHEAD) {
                load_keys(off);
                load_values(off);
            }
        }
        for (; key0 < P.key1; key0 += step) {
            const uint32_t valid = static_cast<uint32_t>(__ballot(off >= 0));
            const bool more = key0 + step < P.key1;
            if (!AHEAD) load_keys(off);
            f32x4 s[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                s[x] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int ks = 0; ks < C::KS; ++ks)
                    s[x] = Mma<T>::run(k_frag<T, C>(kt[x], ks, g, A.D), q[ks], s[x]);
            }
            if (!AHEAD) load_values(off);
            const int64_t off_next = offset_of(key0 + step, page);
            page = page_of(key0 + 2 * step);
            if (AHEAD && more) load_keys(off_next);
            const bool partial = all_see < key0 + kKeys;
            if (valid != 0xffffffffu || partial) mask_scores(s, key0, limit, valid);
            u32x4 pf[1];
            float sum = take_weights<T, C, 1>(R, s, A.scale, pf);
            if (too_much<T>(sum)) sum = move_maximum<T, C, 1>(&R, s, A.scale, pf);
            R.l += sum;
            if (valid != 0xffffffffu) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (!((valid >> ((i >> 2) * 16 + 4 * g + (i & 3))) & 1))
#pragma unroll
                        for (int c = 0; c < C::NC; ++c)
#pragma unroll
                            for (int w = 0; w < C::VW; ++w) vr[i][c].w[w] = 0;
            }
            if (partial && P.seg.causal) {
                bool mine = false;
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int c = 0; c < C::NC; ++c)
#pragma unroll
                        for (int w = 0; w < C::VW; ++w) {
                            const uint32_t x = vr[i][c].w[w];
                            const uint32_t y = C::EB == 2 ? finite_pair<T>(x) : finite_quad(x);
                            mine = mine || x != y;
                            vr[i][c].w[w] = y;
                        }
                if (first_odd < 0 && __any(mine)) first_odd = key0;
            }
#pragma unroll
            for (int j = 0; j < C::NJ; j += 2) {
                u32x4 f[2];
                value_pair(j / C::VE, j % C::VE / 2, &f[0], &f[1]);
                R.o[j] = Mma<T>::run(f[0], pf[0], R.o[j]);
                R.o[j + 1] = Mma<T>::run(f[1], pf[0], R.o[j + 1]);
            }
            if (AHEAD && more) load_values(off_next);
            off = off_next;
        }
        if (first_odd >= 0) {
            // the wave's own steps only: `step` apart
            for (int32_t t = first_odd; t < P.key1; t += step)
                add_not_finite<T, C, false>(A, P.lists, P.pg0, vhd, t,
                                            t + kKeys < P.key1 ? t + kKeys : P.key1, limit, &R);
        }
    }

    // join the waves that shared a head's keys: the upper half of the parts
    // hands over to the lower until one is left
    for (int n = A.kp; n > 1;) {
        const int half = (n + 1) / 2;
        __syncthreads();
        if (works && part >= half && part < n) {
            float* b = lds + ((part - half) * A.hs + h) * (64 * (4 * C::NJ + 2));
            b[lane] = R.m;
            b[64 + lane] = R.l;
#pragma unroll
            for (int j = 0; j < C::NJ; ++j)
                *reinterpret_cast<f32x4*>(b + 128 + (j * 64 + lane) * 4) = R.o[j];
        }
        __syncthreads();
        if (works && part + half < n) {
            const float* b = lds + (part * A.hs + h) * (64 * (4 * C::NJ + 2));
            const float m2 = b[lane], l2 = b[64 + lane];
            const float m = fmaxf(R.m, m2);
            const float ref = m == -INFINITY ? 0.0f : m;
            const float w1 = __builtin_amdgcn_exp2f(R.m - ref), w2 = __builtin_amdgcn_exp2f(m2 - ref);
            R.m = m;
            R.l = R.l * w1 + l2 * w2;
#pragma unroll
            for (int j = 0; j < C::NJ; ++j)
                R.o[j] = R.o[j] * w1 + *reinterpret_cast<const f32x4*>(b + 128 + (j * 64 + lane) * 4) * w2;
        }
        n = half;
    }
    if (works && part == 0) store_rows<T, C, false>(A, to, R, h * kThinRows + a, token, head, live);
    if (A.kp > 1) __syncthreads();
}

// ---------------------------------------------------------------- wide --

// A wide tile's shapes: RT row tiles of 16 per wave, KT keys staged at a time
// in one of two buffers, U steps of 32 computed together.
template <class C>
struct Wide {
    static constexpr int DP = C::KS * 32;
    static constexpr int RT = DP <= 128 ? 2 : 1;
    static constexpr int ROWS = kWaves * 16 * RT;
    static constexpr int KT = DP <= 128 ? 128 : 64;
    static constexpr int U = DP <= 128 ? 2 : 1;
    static constexpr int NB = KT / kKeys;               // steps of 32 keys
    static constexpr int WPG = 128 / KT;                // waves that stage one group of 16 keys
    static constexpr int VR = 16 / WPG;                 // V rows that a wave stages
    static constexpr int KSW = C::KS / WPG;             // k-steps of a K tile that a wave stages
    static constexpr int KF = (KT / 16) * C::KS;        // K fragments of 1 KiB
    static constexpr int RB = DP * 2;                   // bytes of a V row
    static constexpr int BUF = KF * 1024 + KT * RB;
};

typedef __attribute__((address_space(3))) char lds_char;

// 16 bytes per lane from memory to base + 16 * lane of shared memory.
__device__ inline void load_to_lds(const char* src, char* base) {
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) uint32_t*)src,
        (__attribute__((address_space(3))) uint32_t*)base, 16, 0, 0);
}

// V stands in shared memory row by row, its 32-byte pairs of 16-byte chunks
// permuted by row so that the 4 rows x 32 bytes that 16 lanes read together,
// and those of the next 16, lie in different banks.
template <class C>
__device__ inline int v_swizzle(int row) {
    return (C::KS == 2 ? (row >> 1) & 3 : row & 7) << 1;
}

// Operand of the second product for 32 keys from row0 and dims 16 j .. 16 j +
// 15: two transposing reads, each of 4 keys (rows 4 g + 0..3 of a 16-key tile)
// for the lane's dim.
// `at` is v_base's offset; chunk pair j differs from it in the bits of 32 j.
template <class C>
__device__ inline int v_base() {
    const int lane = here_lane(), a = lane & 15, g = lane >> 4;
    const int row = 4 * g + (a >> 2);
    return row * (C::KS * 64) + ((((a >> 1) & 1) ^ v_swizzle<C>(row)) * 16) + (a & 1) * 8;
}

template <class C>
__device__ inline u32x4 v_frag(const char* v, int at, int step, int j) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    constexpr int RB = C::KS * 64;
    const char* p = v + (at ^ (j << 5)) + step * 32 * RB;
    const u32x2 lo = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
    const u32x2 hi = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * RB)));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
}

// Keys [tile0, tile0 + KT) of a piece on their way to a buffer: each wave
// stages K and V of a group of 16 keys, or half of each.  16-bit values go
// from memory to shared memory directly; fp8 ones through registers, where
// they are converted.
template <class T, class C>
struct Stage {
    using W = Wide<C>;
    static constexpr int NK = C::EB == 2 ? 1 : C::NK / W::WPG;            // 16-byte loads per lane
    static constexpr int NV = C::EB == 2 ? 1 : W::VR * W::DP / 1024;
    int64_t off;                        // the row offset of key lane % 16 of the group, or -1
    u32x4 k[NK];
    u32x4 v[NV];
};

// The key whose offset this lane holds, and its page id.
template <class C>
__device__ inline int32_t stage_key(int32_t tile0, int wave) {
    return tile0 + wave / Wide<C>::WPG * 16 + (here_lane() & 15);
}
template <class C>
__device__ inline int32_t stage_page(const Args& A, const Piece& P, int32_t tile0, int wave) {
    return key_page(A, P.lists, P.pg0, stage_key<C>(tile0, wave));
}

template <class T, class C>
__device__ inline void stage_load(const Args& A, Stage<T, C>* S, const char* kh, const char* vhd,
                                  int wave, char* buf, uint32_t* flags) {
    using W = Wide<C>;
    const int lane = here_lane(), g = lane >> 4;
    const int grp = wave / W::WPG, sub = wave % W::WPG;
    const uint64_t seen = __ballot(S->off >= 0);
    const bool whole = seen == ~0ull && A.D == W::DP;       // every lane loads
    if (lane == 0 && sub == 0) reinterpret_cast<uint16_t*>(flags)[grp] = static_cast<uint16_t>(seen);
    const int64_t koff = S->off;                            // of key a, in every lane group
    if constexpr (C::EB == 2) {
        constexpr int LPR = W::RB / 16, RPP = 64 / LPR;     // lanes per V row, rows per load
        constexpr int N = W::VR / RPP;
        int64_t off[N];
#pragma unroll
        for (int i = 0; i < N; ++i) off[i] = __shfl(S->off, sub * W::VR + i * RPP + lane / LPR);
        char* kb = buf + (grp * C::KS + sub * W::KSW) * 1024;
        char* vb = buf + W::KF * 1024 + (grp * 16 + sub * W::VR) * W::RB;
        const char* ksrc = kh + koff + g * 16 + sub * W::KSW * 64;
        if (whole) {
#pragma unroll
            for (int ks = 0; ks < W::KSW; ++ks) load_to_lds(ksrc + ks * 64, kb + ks * 1024);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int row = sub * W::VR + i * RPP + lane / LPR;
                load_to_lds(vhd + off[i] + ((lane % LPR) ^ v_swizzle<C>(row)) * 16, vb + i * 1024);
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < W::KSW; ++ks) {
                if (koff >= 0 && (sub * W::KSW + ks) * 32 + g * 8 < A.D)
                    load_to_lds(ksrc + ks * 64, kb + ks * 1024);
                else
                    *reinterpret_cast<u32x4*>(kb + ks * 1024 + lane * 16) = u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int chunk = (lane % LPR) ^ v_swizzle<C>(sub * W::VR + i * RPP + lane / LPR);
                if (off[i] >= 0 && chunk * 8 < A.D)
                    load_to_lds(vhd + off[i] + chunk * 16, vb + i * 1024);
                else
                    *reinterpret_cast<u32x4*>(vb + i * 1024 + lane * 16) = u32x4{0, 0, 0, 0};
            }
        }
    } else {
        using St = Stage<T, C>;
        constexpr int LPR = W::DP / 16, RPP = 64 / LPR;
#pragma unroll
        for (int y = 0; y < St::NK; ++y) {
            const int b = (sub * St::NK + y) * 64 + g * 16;
            S->k[y] = u32x4{0, 0, 0, 0};
            if (koff >= 0 && b < A.D) S->k[y] = *reinterpret_cast<const u32x4*>(kh + koff + b);
        }
#pragma unroll
        for (int i = 0; i < St::NV; ++i) {
            const int64_t off = __shfl(S->off, sub * W::VR + i * RPP + lane / LPR);
            const int b = lane % LPR * 16;
            S->v[i] = u32x4{0, 0, 0, 0};
            if (off >= 0 && b < A.D) S->v[i] = *reinterpret_cast<const u32x4*>(vhd + off + b);
        }
    }
}

// 8 fp8 values as 8 of the query's type.
template <class T>
__device__ inline u32x4 widen(uint32_t lo, uint32_t hi) {
    return u32x4{Mma<T>::template from_fp8<false>(lo), Mma<T>::template from_fp8<true>(lo),
                 Mma<T>::template from_fp8<false>(hi), Mma<T>::template from_fp8<true>(hi)};
}

template <class T, class C>
__device__ inline void stage_store(const Stage<T, C>& S, int wave, char* buf) {
    if constexpr (C::EB == 1) {
        using W = Wide<C>;
        using St = Stage<T, C>;
        const int lane = here_lane();
        const int grp = wave / W::WPG, sub = wave % W::WPG;
        char* to = buf + (grp * C::KS + sub * W::KSW) * 1024 + lane * 16;
#pragma unroll
        for (int x = 0; x < St::NK; ++x) {
            *reinterpret_cast<u32x4*>(to + 2 * x * 1024) = widen<T>(S.k[x].x, S.k[x].y);
            *reinterpret_cast<u32x4*>(to + (2 * x + 1) * 1024) = widen<T>(S.k[x].z, S.k[x].w);
        }
        constexpr int LPR = W::DP / 16, RPP = 64 / LPR;
        char* v = buf + W::KF * 1024 + grp * 16 * W::RB;
#pragma unroll
        for (int i = 0; i < St::NV; ++i) {
            const int row = sub * W::VR + i * RPP + lane / LPR;
            char* at = v + row * W::RB;
            const int c = 2 * (lane % LPR), sw = v_swizzle<C>(row);
            *reinterpret_cast<u32x4*>(at + ((c ^ sw) * 16)) = widen<T>(S.v[i].x, S.v[i].y);
            *reinterpret_cast<u32x4*>(at + (((c + 1) ^ sw) * 16)) = widen<T>(S.v[i].z, S.v[i].w);
        }
    }
}

template <class T, class C>
struct WideState {
    using W = Wide<C>;
    int32_t limit[W::RT];
    u32x4 q[W::RT][C::KS];
    Rows<C> R[W::RT];
    int32_t most, all_see;
    int32_t first_odd;                  // first tile that values were taken out of, or -1
};

// Clears the infinities and NaN in a wave's eighth of a buffer's V rows; whether there were any.
template <class T, class C>
__device__ inline bool take_out_not_finite(char* buf, int wave) {
    using W = Wide<C>;
    constexpr int N = W::KT * W::RB / kWaves / 1024;
    char* v = buf + W::KF * 1024 + wave * (N * 1024) + here_lane() * 16;
    bool mine = false;
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        u32x4 x = *reinterpret_cast<const u32x4*>(v + i * 1024);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const uint32_t w = finite_pair<T>(x[y]);
            mine = mine || w != x[y];
            x[y] = w;
        }
        *reinterpret_cast<u32x4*>(v + i * 1024) = x;
    }
    return __any(mine);
}

// Orders a block of products and the shared memory reads of their operands: N
// groups of PRODUCTS products, the READS reads of each a group ahead of them
// (left to itself the compiler asks for an operand and waits for it).
template <int N, int READS, int PRODUCTS>
__device__ inline void read_ahead() {
    __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i + 1 < N) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, PRODUCTS, 0);
    }
}

// Steps [from, to) of one buffer against the wave's rows, U steps of 32 keys at a time.
template <class T, class C>
__device__ inline void wide_tile(const Args& A, WideState<T, C>* S, int32_t tile0,
                                 const char* buf, const uint32_t* flags, int from, int to) {
    using W = Wide<C>;
    constexpr int U = W::U;
    const char* v = buf + W::KF * 1024;
    const int lane = here_lane();
    const int vb = v_base<C>();
#pragma unroll 1
    for (int b = from; b < to; b += U) {
        const int32_t key0 = tile0 + b * kKeys;
        if (key0 >= S->most) break;
        bool masked = S->all_see < key0 + U * kKeys;            // some row does not see some key
        uint32_t valid[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            valid[u] = __builtin_amdgcn_readfirstlane(flags[b + u]);
            masked = masked || valid[u] != 0xffffffffu;
        }
        f32x4 s[W::RT][2 * U];
#pragma unroll
        for (int x = 0; x < 2 * U; ++x) {
#pragma unroll
            for (int t = 0; t < W::RT; ++t) s[t][x] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int ks = 0; ks < C::KS; ++ks) {
                const u32x4 f = *reinterpret_cast<const u32x4*>(
                    buf + (((b * 2 + x) * C::KS + ks) * 64 + lane) * 16);
#pragma unroll
                for (int t = 0; t < W::RT; ++t) s[t][x] = Mma<T>::run(f, S->q[t][ks], s[t][x]);
            }
        }
        read_ahead<2 * U, C::KS, C::KS * W::RT>();
        if (masked) {
#pragma unroll
            for (int t = 0; t < W::RT; ++t)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    mask_scores(&s[t][2 * u], key0 + u * kKeys, S->limit[t], valid[u]);
        }
        u32x4 pf[W::RT][U];
#pragma unroll
        for (int t = 0; t < W::RT; ++t) {
            float sum = take_weights<T, C, U>(S->R[t], s[t], A.scale, pf[t]);
            if (__builtin_expect(too_much<T>(sum), 0))
                sum = move_maximum<T, C, U>(&S->R[t], s[t], A.scale, pf[t]);
            S->R[t].l += sum;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < C::NJ; ++j) {
                const u32x4 f = v_frag<C>(v, vb, b + u, j);
#pragma unroll
                for (int t = 0; t < W::RT; ++t) S->R[t].o[j] = Mma<T>::run(f, pf[t][u], S->R[t].o[j]);
            }
        read_ahead<U * C::NJ / 4, 8, 4 * W::RT>();
    }
}

// flags: [2][NB] words, a bit per key that is there; odds: a word per wave.
template <class T, class C>
__device__ void run_wide(const Args& A, const Piece& P, const Dest& to, char* buf0, char* buf1,
                         uint32_t* flags, uint32_t* odds) {
    using W = Wide<C>;
    const int a = here_lane() & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t kvh = P.set;
    count_skipped(A, P, wave);

    const char* kh = A.k + kvh * A.head_stride;
    const char* vhd = A.v + kvh * A.head_stride;
    Stage<T, C> next;
    int32_t page = stage_page<C>(A, P, P.key0, wave);
    next.off = page_offset(A, P.lists, P.pg0, page, stage_key<C>(P.key0, wave), P.key1);
    page = stage_page<C>(A, P, P.key0 + W::KT, wave);
    stage_load<T, C>(A, &next, kh, vhd, wave, buf0, flags);

    WideState<T, C> S;
    const int32_t at = P.tile * A.wide_tokens, past = P.seg.keys - P.seg.ntok;
    const int32_t first = at + wave * 16 * W::RT / A.G;     // this wave's first and last token
    int32_t last = at + (wave * 16 * W::RT + 16 * W::RT - 1) / A.G;
    if (last > P.seg.ntok - 1) last = P.seg.ntok - 1;
    // keys that some row of this wave sees, and that every one does
    S.most = S.all_see = P.key1;
    S.first_odd = -1;
    if (P.seg.causal) {
        if (past + last + 1 < S.most) S.most = past + last + 1;
        S.all_see = past + first + 1;
    }
    if (first >= P.seg.ntok) S.most = 0;                    // no rows
    auto row_of = [&](int t, int32_t* local, int32_t* head) {
        const int row = (wave * W::RT + t) * 16 + a;
        *local = at + row / A.G;
        *head = kvh * A.G + row % A.G;
        return row < A.wide_tokens * A.G && *local < P.seg.ntok;
    };
#pragma unroll
    for (int t = 0; t < W::RT; ++t) {
        int32_t local, head;
        const bool live = row_of(t, &local, &head);
        S.limit[t] = P.key1;
        if (live && P.seg.causal && past + local + 1 < S.limit[t]) S.limit[t] = past + local + 1;
        load_q<T, C>(A, S.q[t], P.seg.tok0 + local, head, live);
        clear(&S.R[t]);
    }

    stage_store<T, C>(next, wave, buf0);
    __syncthreads();
    // one tile: the next one is on its way to the other buffer meanwhile
    auto turn = [&](int32_t tile0, char* here, char* there, uint32_t* fh, uint32_t* ft) {
        const bool more = tile0 + W::KT < P.key1;
        // half of the waves ask for the next tile before the first of their
        // steps, half after it: the memory pipe takes the loads at one rate
        // anyway, and the two waves of a SIMD then run their products and
        // their exponentials at different times
        auto stage_next = [&]() {
            next.off = page_offset(A, P.lists, P.pg0, page, stage_key<C>(tile0 + W::KT, wave), P.key1);
            page = stage_page<C>(A, P, tile0 + 2 * W::KT, wave);
            stage_load<T, C>(A, &next, kh, vhd, wave, there, ft);
        };
        if (more && wave < kWaves / 2) stage_next();
        // where some row of the workgroup does not see some key, values that are
        // not finite leave the buffer (see add_not_finite); once some have, the
        // piece's later ones are added whatever they are
        if (P.seg.causal && tile0 + W::KT > past + at + 1) {
            const bool mine = take_out_not_finite<T, C>(here, wave);
            if ((threadIdx.x & 63) == 0) odds[wave] = mine ? 1u : 0u;
            __syncthreads();
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) any |= odds[w];
            if (S.first_odd < 0 && __builtin_amdgcn_readfirstlane(any) != 0) S.first_odd = tile0;
        }
        wide_tile<T, C>(A, &S, tile0, here, fh, 0, W::U);
        if (more && wave >= kWaves / 2) stage_next();
        wide_tile<T, C>(A, &S, tile0, here, fh, W::U, W::NB);
        if (more) stage_store<T, C>(next, wave, there);
        __syncthreads();
    };
    for (int32_t tile0 = P.key0; tile0 < P.key1; tile0 += 2 * W::KT) {
        turn(tile0, buf0, buf1, flags, flags + W::NB);
        if (tile0 + W::KT < P.key1) turn(tile0 + W::KT, buf1, buf0, flags + W::NB, flags);
    }
    if (S.first_odd >= 0) {
#pragma unroll
        for (int t = 0; t < W::RT; ++t)
            add_not_finite<T, C, true>(A, P.lists, P.pg0, vhd, S.first_odd, S.most, S.limit[t], &S.R[t]);
    }
#pragma unroll
    for (int t = 0; t < W::RT; ++t) {
        int32_t local, head;
        const bool live = row_of(t, &local, &head);
        store_rows<T, C, true>(A, to, S.R[t], (wave * W::RT + t) * 16 + a, P.seg.tok0 + local, head,
                               live);
    }
}

// -------------------------------------------------------------- kernel --

__device__ inline int64_t wave_scan(int64_t x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    return x;
}

constexpr int kWindow = 64;     // segments whose values are held in shared memory

struct Plan {
    int64_t sums[kWaves][2];    // per-wave totals of a chunk
    int64_t at[2];              // {segment, its start} of this workgroup's first unit
    Seg seg[kWindow];           // a window of segments
    int64_t pg0[kWindow];
    int64_t units[kWindow];     // of a head set
};

// The workgroup's line (0 thin, 1 wide), its piece [lo, hi) of it and the
// segment that the piece begins in.  Every workgroup scans all segments (512
// at a time); the first one also leaves their starts and the lines' lengths
// for k_attend_join.
struct Mine {
    int line;
    int64_t n, wgs;             // its units and workgroups
    int64_t w, lo, hi;
    int64_t slot0;              // the line's first slot
    int32_t seg;
    int32_t window;             // first segment of the window in shared memory
    int64_t seg_start;
};

template <int LINES>
__device__ inline Mine plan_work(const Args& A, Plan* L, uint32_t block, uint32_t grid) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t nseg = A.num_groups + A.num_reqs;
    int64_t total[2] = {0, 0};
    int64_t start = 0, cost = 0;            // of this thread's segment in the last chunk
    bool wide = false;
    Seg mine = {};
    int64_t units = 0, pg0 = 0;
    for (int32_t c0 = 0; c0 < nseg; c0 += kThreads) {
        const int32_t s = c0 + static_cast<int32_t>(threadIdx.x);
        cost = 0;
        wide = false;
        if (s < nseg) {
            pg0 = s < A.num_groups ? A.pre.pg_off[s] : A.own.pg_off[s - A.num_groups];
            mine = segment(A, s);
            units = set_units(mine);
            cost = units * mine.sets;
            wide = (LINES & 2) && mine.wide;
        }
        const int64_t x = LINES & 1 ? wave_scan(wide ? 0 : cost) : 0;
        const int64_t y = LINES & 2 ? wave_scan(wide ? cost : 0) : 0;
        if (lane == 63) {
            L->sums[wave][0] = x;
            L->sums[wave][1] = y;
        }
        __syncthreads();
        int64_t before[2] = {total[0], total[1]};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            const int64_t sx = L->sums[v][0], sy = L->sums[v][1];
            if (v < wave) { before[0] += sx; before[1] += sy; }
            total[0] += sx;
            total[1] += sy;
        }
        start = wide ? before[1] + y - cost : before[0] + x - cost;
        if (block == 0 && s < nseg) A.placed[s] = Placed{mine, start, units};
        if (c0 + kThreads < nseg) __syncthreads();
    }
    total[0] = uniform(total[0]);
    total[1] = uniform(total[1]);

    // workgroups per line: by the lines' times, in eights (one per XCD), and
    // no more than keep a piece at its least length
    int64_t share = 0;                      // workgroups of the wide line
    if (total[1] > 0) {
        share = grid;
        if (total[0] > 0) {
            const float tw = static_cast<float>(total[1]) * A.wide_weight;
            const float tt = static_cast<float>(total[0]);
            share = static_cast<int64_t>(grid * (tw / (tw + tt)) / 8.0f + 0.5f) * 8;
            share = clamp_to(share, 8, static_cast<int64_t>(grid) - 8);
        }
    }
    int64_t wgs[2] = {static_cast<int64_t>(grid) - share, share};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int log2 = i ? A.wide_min_log2 : A.thin_min_log2;
        const int64_t want = (((total[i] + (int64_t(1) << log2) - 1) >> log2) + 7) / 8 * 8;
        wgs[i] = uniform(wgs[i] > want ? want : wgs[i]);
    }
    if (block == 0 && threadIdx.x == 0) {
        const Cuts thin(total[0], wgs[0]), wide_cuts(total[1], wgs[1]);
        A.plan[0] = thin.q;
        A.plan[1] = thin.r;
        A.plan[2] = wide_cuts.q;
        A.plan[3] = wide_cuts.r;
        A.plan[4] = wgs[0];
        A.plan[5] = wgs[1];
    }
    // consecutive pieces on one XCD (workgroups are dealt to the eight in turn)
    Mine M;
    const int64_t xcd = block % 8, j = block / 8;
    M.line = j < wgs[1] / 8 ? 1 : 0;
    M.slot0 = M.line ? 0 : 2 * wgs[1];
    const int64_t all = M.line ? wgs[1] : wgs[0];
    const int64_t jj = M.line ? j : j - wgs[1] / 8;
    M.w = xcd * (all / 8) + jj;
    M.lo = M.hi = 0;
    if (jj >= all / 8) return M;
    if (threadIdx.x == 0) A.splits[M.slot0 / 2 + M.w].last = -1;
    M.n = M.line ? total[1] : total[0];
    M.wgs = all;
    const Cuts cuts(M.n, all);
    M.lo = uniform(cuts.start(M.w));
    M.hi = uniform(cuts.start(M.w + 1));
    if (M.lo >= M.hi) return M;
    // the segment that unit lo lies in
    if (nseg > kThreads) {
        __syncthreads();
        int64_t run = 0;
        for (int32_t c0 = 0; c0 < nseg; c0 += kThreads) {
            const int32_t s = c0 + static_cast<int32_t>(threadIdx.x);
            int64_t cc = 0;
            if (s < nseg) {
                const Seg g = segment(A, s);
                if (g.wide == (M.line == 1)) cc = set_units(g) * g.sets;
            }
            const int64_t x = wave_scan(cc);
            if (lane == 63) L->sums[wave][0] = x;
            __syncthreads();
            int64_t before = run;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                if (v < wave) before += L->sums[v][0];
                run += L->sums[v][0];
            }
            const int64_t b = before + x - cc;
            if (cc > 0 && b <= M.lo && M.lo < b + cc) {
                L->at[0] = s;
                L->at[1] = b;
            }
            __syncthreads();
            if (uniform(run) > M.lo) break;
        }
    } else {
        if (cost > 0 && wide == (M.line == 1) && start <= M.lo && M.lo < start + cost) {
            L->at[0] = threadIdx.x;
            L->at[1] = start;
        }
        __syncthreads();
    }
    M.seg = uniform(static_cast<int32_t>(L->at[0]));
    M.seg_start = uniform(L->at[1]);
    M.window = M.seg - kWindow;
    if (nseg <= kThreads) {                 // the window is at hand
        const int32_t i = static_cast<int32_t>(threadIdx.x) - M.seg;
        if (i >= 0 && i < kWindow) {
            L->seg[i] = mine;
            L->units[i] = units;
            L->pg0[i] = pg0;
        }
        M.window = M.seg;
        __syncthreads();
    }
    return M;
}

// LINES: 1 thin, 2 wide, 3 both.
template <class T, bool FP8, int DP, int LINES>
struct Shared {
    using C = Cfg<T, FP8, DP>;
    static constexpr int THIN = LINES & 1 ? (kWaves / 2) * 64 * (4 * C::NJ + 2) * 4 : 16;
    static constexpr int BUF = LINES == 1 ? 16 : Wide<C>::BUF;
    static constexpr int BUF0 = BUF > THIN ? BUF : THIN;
};

template <class T, bool FP8, int DP, int LINES>
__global__ __launch_bounds__(kThreads, 2) void k_attend(const Args A) {
    using C = Cfg<T, FP8, DP>;
    using S = Shared<T, FP8, DP, LINES>;
    __shared__ Plan plan;
    // separate arrays: reads of one need not wait for loads on their way to the other
    __shared__ __attribute__((aligned(16))) char buf0[S::BUF0];
    __shared__ __attribute__((aligned(16))) char buf1[S::BUF];
    __shared__ uint32_t flags[2 * Wide<C>::NB];
    __shared__ uint32_t odds[kWaves];
    const Mine M = plan_work<LINES>(A, &plan, blockIdx.x, gridDim.x);
    if (M.lo >= M.hi) return;
    const bool wide_line = LINES == 2 || (LINES == 3 && M.line == 1);
    const int32_t nseg = A.num_groups + A.num_reqs;
    const int step_log2 = wide_line ? (Wide<C>::KT == 128 ? 7 : 6) : 5;

    Piece P;
    int64_t pos = M.lo;                     // on the line
    int32_t s = M.seg, first = M.window;
    int64_t seg_start = M.seg_start;
    while (pos < M.hi && s < nseg) {
        if (s >= first + kWindow) {
            first = s;
            __syncthreads();
            const int32_t t = first + static_cast<int32_t>(threadIdx.x);
            if (threadIdx.x < kWindow && t < nseg) {
                const Seg g = segment(A, t);
                plan.seg[threadIdx.x] = g;
                plan.units[threadIdx.x] = set_units(g);
                plan.pg0[threadIdx.x] = t < A.num_groups ? A.pre.pg_off[t] : A.own.pg_off[t - A.num_groups];
            }
            __syncthreads();
        }
        P.seg = uniform(plan.seg[s - first]);
        const int64_t per_set = uniform(plan.units[s - first]);
        const int64_t cost = per_set * P.seg.sets;
        if (cost == 0 || P.seg.wide != (M.line == 1)) { ++s; continue; }
        const bool pre = s < A.num_groups;
        P.lists = pre ? A.pre : A.own;
        P.pg0 = uniform(plan.pg0[s - first]);
        while (pos < M.hi && pos < seg_start + cost) {
            const int64_t x = pos - seg_start;
            P.set = P.seg.sets == 1 ? 0 : static_cast<int32_t>(x / per_set);
            const int64_t y = x - P.set * per_set;
            // the tile that unit y of the head set lies in
            int32_t lo = 0, hi = P.seg.tiles - 1;
            if (hi > 0) {
                if (!P.seg.causal) {
                    lo = static_cast<int32_t>(y / (static_cast<int64_t>(P.seg.base) + P.seg.extra));
                } else {
                    while (lo < hi) {
                        const int32_t mid = lo + (hi - lo + 1) / 2;
                        if (tile_start(P.seg, mid) <= y) lo = mid; else hi = mid - 1;
                    }
                }
            }
            P.tile = lo;
            const int64_t keys = tile_keys(P.seg, lo), len = keys + P.seg.extra;
            const int64_t item = seg_start + P.set * per_set + tile_start(P.seg, lo);
            const int64_t end = M.hi < item + len ? M.hi : item + len;
            const bool from_start = pos == item, to_end = end == item + len;
            // cuts inside an item fall on whole steps, both sides alike
            const int32_t seen = static_cast<int32_t>(keys < P.seg.keys ? keys : P.seg.keys);
            P.key0 = cut_key(P.seg, pos - item, step_log2, seen);
            P.key1 = to_end ? seen : cut_key(P.seg, end - item, step_log2, seen);
            P.counts = P.set == 0 && P.tile == P.seg.tiles - 1;
            Dest to;
            if (from_start && to_end) {
                to.kind = A.num_groups > 0 ? kRowBuffer : kFinal;
            } else {
                to.kind = kSlot;
            }
            to.part = pre ? 1 : 0;
            to.slot = static_cast<int32_t>(M.slot0 + 2 * M.w + (from_start ? 1 : 0));
            pos = end;
            if (!to_end && threadIdx.x == 0) {
                const Cuts cuts(M.n, M.wgs);
                Split x;
                x.item = item;
                x.last = static_cast<int32_t>(cuts.piece_of(item + len - 1));
                x.w = static_cast<int32_t>(cuts.piece_of(item));
                x.slot0 = static_cast<int32_t>(M.slot0);
                x.wide = wide_line;
                x.tok0 = P.seg.tok0;
                x.ntok = P.seg.ntok;
                x.set = P.set;
                x.tile = P.tile;
                x.keys = seen;
                x.extra = P.seg.extra;
                A.splits[M.slot0 / 2 + M.w] = x;
            }
            // a piece without a step of its own leaves nothing (k_attend_join sees it the same way)
            if (to.kind == kSlot && P.key0 >= P.key1) continue;
            if constexpr (LINES & 2) {
                if (wide_line) run_wide<T, C>(A, P, to, buf0, buf1, flags, odds);
            }
            if constexpr (LINES & 1) {
                if (!wide_line) run_thin<T, C>(A, P, to, reinterpret_cast<float*>(buf0));
            }
        }
        seg_start += cost;
        ++s;
    }
}

// ---------------------------------------------------------------- join --

// The list entry r with off[r] <= x < off[r + 1] (off non-decreasing, n lists),
// by a 64-way search of the wave.
__device__ inline int32_t find_list(const int64_t* off, int32_t n, int64_t x) {
    const int lane = threadIdx.x & 63;
    int32_t lo = 0, len = n;                // the answer is in [lo, lo + len)
    while (len > 1) {
        const int32_t step = (len + 63) / 64;
        const int32_t at = lo + lane * step;
        const uint64_t below = __ballot(lane * step < len && off[at < n ? at : n] <= x);
        const int32_t k = below == 0 ? 0 : 63 - __clzll(below);
        const int32_t rest = len - k * step;
        lo += k * step;
        len = rest < step ? rest : step;
    }
    return lo;
}

// Partial sums of one row under way: lane holds 4 dims of it.
struct Sum {
    float m, l;
    f32x4 o;
    __device__ inline Sum() : m(-INFINITY), l(0.0f), o{0, 0, 0, 0} {}
    __device__ inline void add(float2 ml, f32x4 x) {
        if (ml.y == 0.0f) return;
        const float top = fmaxf(m, ml.x);
        const float ref = top == -INFINITY ? 0.0f : top;
        const float w1 = __builtin_amdgcn_exp2f(m - ref), w2 = __builtin_amdgcn_exp2f(ml.x - ref);
        m = top;
        l = l * w1 + ml.y * w2;
        o = o * w1 + x * w2;
    }
    template <class T>
    __device__ inline void store(const Args& A, int32_t token, int32_t head, int d) const {
        const float inv = l == 0.0f ? 0.0f : A.v_scale / l;
        if (d < A.D)
            *reinterpret_cast<u32x2*>(A.out + static_cast<int64_t>(token) * A.out_stride +
                                      (static_cast<int64_t>(head) * A.D + d) * 2) =
                u32x2{Mma<T>::pack(o[0] * inv, o[1] * inv), Mma<T>::pack(o[2] * inv, o[3] * inv)};
        if (d == 0 && A.lse != nullptr)
            A.lse[static_cast<int64_t>(token) * A.H * A.G + head] =
                l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
    }
};

// Adds row `slot_row` of the pieces w0 + way, w0 + way + ways .. w1 of an item
// that begins at unit `item`; a workgroup has left its slot if its piece has a
// step of keys.
__device__ inline void add_slots(const Args& A, Sum* sum, const Seg& g, const Cuts& cuts, int64_t item,
                                 int32_t keys, int32_t w0, int32_t w1, int32_t slot0, int slot_row,
                                 int d, int step_log2, int way, int ways) {
    constexpr int B = 4;                    // slots under way at once
    for (int32_t w = w0 + way; w <= w1; w += B * ways) {
        float2 ml[B];
        f32x4 x[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            ml[i] = make_float2(0.0f, 0.0f);
            x[i] = f32x4{0, 0, 0, 0};
            const int32_t v = w + i * ways;
            if (v > w1) continue;
            const int32_t k0 = v == w0 ? 0 : cut_key(g, cuts.start(v) - item, step_log2, keys);
            const int32_t k1 = v == w1 ? keys : cut_key(g, cuts.start(v + 1) - item, step_log2, keys);
            if (k0 >= k1) continue;
            const int64_t at = static_cast<int64_t>(slot0 + 2 * v + (v == w0 ? 1 : 0)) * A.slot_rows + slot_row;
            ml[i] = *reinterpret_cast<const float2*>(A.slot_ml + at * 2);
            if (d < A.D) x[i] = *reinterpret_cast<const f32x4*>(A.slot_o + at * A.D + d);
        }
#pragma unroll
        for (int i = 0; i < B; ++i) sum->add(ml[i], x[i]);
    }
}

// The sums of `ways` neighbouring waves, in the first of them, in the order of
// the waves.
__device__ inline void join_ways(Sum* sum, float (*lds)[6][64], int wave, int way, int ways) {
    if (ways == 1) return;
    const int lane = threadIdx.x & 63;
    __syncthreads();                        // the last rows' sums are read
    if (way > 0) {
        lds[wave][0][lane] = sum->m;
        lds[wave][1][lane] = sum->l;
#pragma unroll
        for (int i = 0; i < 4; ++i) lds[wave][2 + i][lane] = sum->o[i];
    }
    __syncthreads();
    if (way > 0) return;
#pragma unroll 1
    for (int w = wave + 1; w < wave + ways; ++w)
        sum->add(make_float2(lds[w][0][lane], lds[w][1][lane]),
                 f32x4{lds[w][2][lane], lds[w][3][lane], lds[w][4][lane], lds[w][5][lane]});
}

// Without prefixes: an item that lies in n pieces is joined by kJoinParts
// workgroups for each of the first n - 1, its rows dealt to their waves; with
// many pieces, `ways` waves share a row's.  (One wave for all pieces of a row
// took 26 us for 4 requests behind 2048 tokens, most of the call.)  Workgroups
// behind those write the rows of requests without keys, 64 requests a wave.
template <class T, int DP>
__global__ __launch_bounds__(64 * kJoinWaves) void k_attend_join_items(const Args A, int32_t pieces) {
    constexpr int LPR = DP / 4, RPW = 64 / LPR;
    __shared__ float sums[kJoinWaves][6][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int d = lane % LPR * 4, sub_row = lane / LPR;
    const int32_t hq = A.H * A.G;
    const int32_t block = blockIdx.x;
    if (block >= pieces * kJoinParts) {
        const int32_t r0 = ((block - pieces * kJoinParts) * kJoinWaves + wave) * 64;
        int32_t t0 = 0, n = 0;
        if (r0 + lane < A.num_reqs && A.ctx[r0 + lane] <= 0) {
            t0 = clamp_to(A.tok_off[r0 + lane], 0, A.T);
            n = clamp_to(A.tok_off[r0 + lane + 1], t0, A.T) - t0;
        }
        for (uint64_t todo = __ballot(n > 0); todo != 0; todo &= todo - 1) {
            const int who = __ffsll(static_cast<unsigned long long>(todo)) - 1;
            const int64_t rows = static_cast<int64_t>(__shfl(n, who)) * hq;
            const int32_t first = __shfl(t0, who);
            for (int64_t x = sub_row; x < rows; x += RPW)
                Sum().store<T>(A, first + static_cast<int32_t>(x / hq), static_cast<int32_t>(x % hq), d);
        }
        return;
    }
    const int32_t piece = block / kJoinParts;
    const Split S = A.splits[piece];
    if (piece >= A.plan[4] + A.plan[5] || S.last < 0) return;
    const int32_t n = uniform(S.last - S.w);            // pieces less one
    const int ways = n < 4 ? 1 : (n < 8 ? 2 : (n < 16 ? 4 : 8));
    const int way = wave % ways, teams = kJoinWaves / ways;
    const int32_t me = uniform((piece - S.slot0 / 2 - S.w) * kJoinParts) + block % kJoinParts;
    Cuts cuts;
    cuts.q = A.plan[S.wide ? 2 : 0];
    cuts.r = A.plan[S.wide ? 3 : 1];
    Seg g;
    g.extra = S.extra;
    const int step_log2 = S.wide ? (DP <= 128 ? 7 : 6) : 5;
    const int rows = uniform(S.wide ? A.wide_tokens * A.G : A.hs * kThinRows);
    for (int row0 = me * teams * RPW; row0 < rows; row0 += kJoinParts * n * teams * RPW) {
        const int row = row0 + wave / ways * RPW + sub_row;
        int32_t local, head;
        bool live = row < rows;
        if (S.wide) {
            local = S.tile * A.wide_tokens + row / A.G;
            head = S.set * A.G + row % A.G;
        } else {
            const int a = row % kThinRows;
            const int32_t vh = S.set * A.hs + row / kThinRows;
            const int32_t kvh = vh / A.parts, hin = vh % A.parts * A.gv + a % A.gv;
            local = S.tile * A.thin_tokens + a / A.gv;
            head = kvh * A.G + hin;
            live = live && a < A.thin_tokens * A.gv && kvh < A.H && hin < A.G;
        }
        live = live && local < S.ntok;
        Sum sum;
        if (live)
            add_slots(A, &sum, g, cuts, S.item, S.keys, S.w, S.last, S.slot0, row, d, step_log2, way, ways);
        join_ways(&sum, sums, wave, way, ways);
        if (live && way == 0) sum.store<T>(A, S.tok0 + local, head, d);
    }
}

// With prefixes: the workgroups (x, .) join the rows of token x, each from its
// two parts, a thin head's query heads (256 / DP of them) by `ways` waves.
// Bound by its launch and its dependent loads: the lists that the token is in
// (guessed for one token per request, searched for otherwise), then the parts.
template <class T, int DP, bool SHARED>
__global__ __launch_bounds__(64 * kJoinWaves) void k_attend_join(const Args A, int32_t many) {
    const int32_t ways = SHARED ? many : 1;
    constexpr int LPR = DP / 4, RPW = 64 / LPR;
    __shared__ float sums[kJoinWaves][6][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t token = blockIdx.x;
    const int d = lane % LPR * 4;

    int32_t r = token < A.num_reqs ? token : A.num_reqs - 1;
    Placed part[2] = {A.placed[A.num_groups + r], A.placed[0]};
    Cuts thin, wide;
    thin.q = uniform(A.plan[0]);
    thin.r = uniform(A.plan[1]);
    wide.q = uniform(A.plan[2]);
    wide.r = uniform(A.plan[3]);
    const int32_t wgs1 = uniform(static_cast<int32_t>(A.plan[5]));
    if (uniform(static_cast<int32_t>(token < part[0].g.tok0 || token >= part[0].g.tok0 + part[0].g.ntok))) {
        r = uniform(find_list(A.tok_off, A.num_reqs, token));
        part[0] = A.placed[A.num_groups + r];
        const int32_t end = part[0].g.tok0 + part[0].g.ntok;
        if (uniform(static_cast<int32_t>(token >= end)) != 0) return;      // behind the last request
    }
    if (A.num_groups > 1) part[1] = A.placed[uniform(find_list(A.grp_off, A.num_groups, r))];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        part[k].g = uniform(part[k].g);
        part[k].start = uniform(part[k].start);
        part[k].units = uniform(part[k].units);
    }

    const int32_t per = (A.gv + RPW - 1) / RPW, units = A.H * A.parts * per;
    {
        const int32_t way = wave % ways, mine = (blockIdx.y * kJoinWaves + wave) / ways;
        const bool works = mine < units;
        const int32_t u = works ? mine : 0;
        const int32_t vh = u / per, kvh = vh / A.parts, sub = vh - kvh * A.parts;
        const int32_t in = (u - vh * per) * RPW + lane / LPR, hin = sub * A.gv + in;
        const bool live = works && in < A.gv && hin < A.G;
        const int32_t head = kvh * A.G + (live ? hin : 0);
        const int64_t row = static_cast<int64_t>(token) * A.H * A.G + head;
        Sum sum;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Seg& g = part[k].g;
            const int32_t local = token - g.tok0;
            if (!works || g.tiles == 0 || local < 0 || local >= g.ntok) continue;
            const Cuts& cuts = g.wide ? wide : thin;
            const int32_t tile = local / g.tp, in_tile = local - tile * g.tp;
            const int32_t set = g.wide ? kvh : vh / A.hs;
            const int64_t item = part[k].start + set * part[k].units + tile_start(g, tile);
            const int64_t keys = tile_keys(g, tile);
            const int32_t w0 = static_cast<int32_t>(cuts.piece_of(item));
            if (item + keys + g.extra <= cuts.start(w0 + 1)) {     // one workgroup had it all
                if (way > 0) continue;
                const int64_t at = static_cast<int64_t>(k) * A.T * A.H * A.G + row;
                const float2 ml = *reinterpret_cast<const float2*>(A.row_ml + at * 2);
                sum.add(ml, d < A.D ? *reinterpret_cast<const f32x4*>(A.row_o + at * A.D + d) : f32x4{0, 0, 0, 0});
            } else {
                const int32_t w1 = static_cast<int32_t>(cuts.piece_of(item + keys + g.extra - 1));
                const int slot_row = g.wide ? in_tile * A.G + (live ? hin : 0)
                                            : (vh - set * A.hs) * kThinRows + in_tile * A.gv + (live ? in : 0);
                add_slots(A, &sum, g, cuts, item, static_cast<int32_t>(keys < g.keys ? keys : g.keys), w0,
                          w1, g.wide ? 0 : 2 * wgs1, slot_row, d, !g.wide ? 5 : (DP <= 128 ? 7 : 6), way, ways);
            }
        }
        join_ways(&sum, sums, wave, way, ways);
        if (live && way == 0) sum.store<T>(A, token, head, d);
    }
}

}  // namespace attend
}  // namespace kvx
