// kvx_tables.hpp -- page tables and slot maps built from request lengths, and
// new K/V rows written at those slots (gfx950 / CDNA4).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kvx {
namespace tables {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ building --
//
// With a_r = add[r], c_r = have[r] + a_r, P_r = ceil(c_r / B) pages in all and
// h_r = ceil(have[r] / B) held ones, three exclusive sums over the requests
// (of a, P and P - h) give the token offsets, the table offsets and the place
// of each request's new pages in the free list.  The outputs are cut into
// windows of slots and page ids, one workgroup each.  Every workgroup sums the
// requests itself, a chunk at a time, keeps a chunk's sums in shared memory and
// fills the outputs of its window that belong to the chunk, each run of a
// thread found by a binary search there: one launch, no order between
// workgroups, and no request's length makes one workgroup's work longer.
//
// Bound by the chain launch - lengths - sums - search - ids of a workgroup, not
// by bytes.  One slot and one id a thread shorten the chain (a decode step of
// 64 requests 5.5 us against 8.0 with 4 and 2, 32 prompts page by token 5.4
// against 7.5, both with four requests a thread); with many workgroups their
// sums are what counts, and 4 and 2 are faster (2048 requests, 540 thousand
// ids: 18.7 us against 25.3).  The host takes the short runs up to kShortGrid
// workgroups.  Likewise a thread sums one
// request where a chunk of those holds the batch (64 requests 4.5 us against
// 5.5 with four, 256 4.9 against 5.9), and four where not: every chunk is
// another round of the chain (1024 requests 8.3 us against 15.7 with one).
constexpr int kBuildThreads = 256;
constexpr int kLongSlotRun = 4;         // outputs of a thread in a large grid
constexpr int kLongIdRun = 2;
constexpr int64_t kShortGrid = 512;
constexpr int kFewRequests = kBuildThreads;     // one a thread
constexpr int kManyPerThread = 4;

struct BuildArgs {
    const int32_t* have;        // or NULL: none
    const int32_t* add;
    const int64_t* held_off;    // with have
    const int32_t* held_ids;
    int64_t num_held;
    const int32_t* free_ids;
    int64_t num_free;
    int32_t num_reqs;
    int32_t page_size;
    int32_t page_shift;         // log2(page_size), or -1
    int32_t* ctx;
    int64_t* tok_off;
    int64_t* pg_off;
    int32_t* ids;
    int64_t cap_ids;
    int64_t* slots;
    int64_t cap_tokens;
    int64_t* totals;            // or NULL
};

// x / page_size; lengths and their sum with a page size fit 32 bits.
template <class Args>
__device__ inline uint32_t page_index(const Args& A, uint32_t x) {
    return A.page_shift >= 0 ? x >> A.page_shift : x / static_cast<uint32_t>(A.page_size);
}

struct Sums {
    int64_t tok, pg, fresh;
};

__device__ inline Sums operator+(const Sums& a, const Sums& b) {
    return Sums{a.tok + b.tok, a.pg + b.pg, a.fresh + b.fresh};
}

template <int kPerThread>
struct BuildShared {
    static constexpr int kChunk = kBuildThreads * kPerThread;
    int64_t tok[kChunk + 1];
    int64_t pg[kChunk + 1];
    int64_t fresh[kChunk];
    int32_t have[kChunk];
    Sums wave[kBuildThreads / 64];
};

// Largest i of [0, n) with off[i] <= x (off non-decreasing, off[0] <= x).
__device__ inline int last_not_above(const int64_t* off, int n, int64_t x) {
    int lo = 0;
    for (int len = n; len > 1;) {
        const int half = len / 2;
        if (off[lo + half] <= x) lo += half;
        len -= half;
    }
    return lo;
}

// Page k of request r (i-th of the chunk): a held page, or one of the free list; -1 if there is none.
template <class Shared>
__device__ inline int32_t page_of(const BuildArgs& A, const Shared& S, int32_t r, int i, int64_t k) {
    const int64_t held = page_index(A, static_cast<uint32_t>(S.have[i]) + A.page_size - 1);
    if (k < held) {
        const int64_t off = A.held_off[r];
        if (off < -k || off >= A.num_held - k) return -1;
        return A.held_ids[off + k];
    }
    const int64_t at = S.fresh[i] + k - held;
    return at < A.num_free ? A.free_ids[at] : -1;
}

template <int kSlotRun, int kIdRun, int kPerThread>
__global__ __launch_bounds__(kBuildThreads) void k_build_tables(const BuildArgs A) {
    constexpr int kSlotWindow = kBuildThreads * kSlotRun, kIdWindow = kBuildThreads * kIdRun;
    constexpr int kChunk = kBuildThreads * kPerThread;
    __shared__ BuildShared<kPerThread> S;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool first = blockIdx.x == 0;
    const int64_t slot0 = static_cast<int64_t>(blockIdx.x) * kSlotWindow;
    const int64_t id0 = static_cast<int64_t>(blockIdx.x) * kIdWindow;
    const int64_t slot1 = slot0 + kSlotWindow < A.cap_tokens ? slot0 + kSlotWindow : A.cap_tokens;
    const int64_t id1 = id0 + kIdWindow < A.cap_ids ? id0 + kIdWindow : A.cap_ids;
    Sums run{0, 0, 0};
    for (int32_t c0 = 0; c0 < A.num_reqs; c0 += kChunk) {
        Sums mine[kPerThread], sum{0, 0, 0};
        int32_t have[kPerThread];
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int32_t r = c0 + tid * kPerThread + i;
            int64_t h = 0, a = 0;
            if (r < A.num_reqs) {
                if (A.have != nullptr && A.have[r] > 0) h = A.have[r];
                if (A.add[r] > 0) a = A.add[r];
                if (h + a > INT32_MAX) a = INT32_MAX - h;
            }
            have[i] = static_cast<int32_t>(h);
            const uint32_t b = A.page_size;
            const int64_t pages = page_index(A, static_cast<uint32_t>(h + a) + b - 1);
            const int64_t held = page_index(A, static_cast<uint32_t>(h) + b - 1);
            mine[i] = sum;                              // exclusive inside the thread
            sum = sum + Sums{a, pages, pages - held};
        }
        Sums incl = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const Sums y{__shfl_up(incl.tok, d), __shfl_up(incl.pg, d), __shfl_up(incl.fresh, d)};
            if (lane >= d) incl = incl + y;
        }
        if (lane == 63) S.wave[wave] = incl;
        __syncthreads();
        Sums before = run, all = run;
#pragma unroll
        for (int v = 0; v < kBuildThreads / 64; ++v) {
            if (v < wave) before = before + S.wave[v];
            all = all + S.wave[v];
        }
        before = before + Sums{incl.tok - sum.tok, incl.pg - sum.pg, incl.fresh - sum.fresh};
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int j = tid * kPerThread + i;
            const Sums x = before + mine[i];
            S.tok[j] = x.tok;
            S.pg[j] = x.pg;
            S.fresh[j] = x.fresh;
            S.have[j] = have[i];
        }
        if (tid == 0) {
            S.tok[kChunk] = all.tok;
            S.pg[kChunk] = all.pg;
        }
        __syncthreads();
        const int n = A.num_reqs - c0 < kChunk ? A.num_reqs - c0 : kChunk;
        if (first) {
            for (int j = tid; j < n; j += kBuildThreads) {
                A.tok_off[c0 + j] = S.tok[j];
                A.pg_off[c0 + j] = S.pg[j];
                A.ctx[c0 + j] = S.have[j] + static_cast<int32_t>(S.tok[j + 1] - S.tok[j]);
            }
        }
        // runs of neighbouring outputs per thread: one search, then a walk along
        // the chunk's requests; all of a run's table reads are under way at once
        const int64_t s1 = slot1 < all.tok ? slot1 : all.tok;
        for (int64_t x0 = slot0 + tid * kSlotRun; x0 < s1; x0 += kBuildThreads * kSlotRun) {
            if (x0 + kSlotRun <= run.tok) continue;
            const int64_t from = x0 > run.tok ? x0 : run.tok;
            int i = last_not_above(S.tok, n, from);
            int32_t page[kSlotRun];
            uint32_t in_page[kSlotRun];
#pragma unroll
            for (int y = 0; y < kSlotRun; ++y) {
                const int64_t x = x0 + y;
                page[y] = -1;
                if (x < from || x >= s1) continue;
                while (i + 1 < n && S.tok[i + 1] <= x) ++i;
                const uint32_t t = S.have[i] + static_cast<uint32_t>(x - S.tok[i]);
                const uint32_t k = page_index(A, t);
                in_page[y] = t - k * A.page_size;
                page[y] = page_of(A, S, c0 + i, i, k);
            }
#pragma unroll
            for (int y = 0; y < kSlotRun; ++y)
                if (x0 + y >= from && x0 + y < s1)
                    A.slots[x0 + y] = page[y] < 0 ? -1 : static_cast<int64_t>(page[y]) * A.page_size + in_page[y];
        }
        const int64_t p1 = id1 < all.pg ? id1 : all.pg;
        for (int64_t x0 = id0 + tid * kIdRun; x0 < p1; x0 += kBuildThreads * kIdRun) {
            if (x0 + kIdRun <= run.pg) continue;
            const int64_t from = x0 > run.pg ? x0 : run.pg;
            int i = last_not_above(S.pg, n, from);
            int32_t page[kIdRun];
#pragma unroll
            for (int y = 0; y < kIdRun; ++y) {
                const int64_t x = x0 + y;
                if (x < from || x >= p1) continue;
                while (i + 1 < n && S.pg[i + 1] <= x) ++i;
                page[y] = page_of(A, S, c0 + i, i, x - S.pg[i]);
            }
#pragma unroll
            for (int y = 0; y < kIdRun; ++y)
                if (x0 + y >= from && x0 + y < p1) A.ids[x0 + y] = page[y];
        }
        run = all;
        if (!first && run.tok >= slot1 && run.pg >= id1) return;   // the same for every thread
        __syncthreads();
    }
    if (first && tid == 0) {
        A.tok_off[A.num_reqs] = run.tok;
        A.pg_off[A.num_reqs] = run.pg;
        if (A.totals != nullptr) {
            A.totals[0] = run.tok;
            A.totals[1] = run.pg;
            A.totals[2] = run.fresh;
            A.totals[3] = run.fresh > A.num_free ? run.fresh - A.num_free : 0;
        }
    }
}

// ----------------------------------------------------------- appending --
//
// Row t of K and of V goes to slot slots[t] of the layer's planes.  The rows'
// 16-byte pieces are numbered token by token (K's pieces, then V's), one to a
// thread.  Bound by memory: 49152 tokens of 1 KiB rows move at 5.08 TB/s read
// and written (39.7 us); 2, 4 or 8 pieces a thread lose (42.9, 46.3, 48.3 us;
// one decode step of 64 tokens 2.4 us against 2.7, 3.5, 5.0): more workgroups
// hide the slot's load better than more loads per thread.  Sources are read
// past the caches (46.5 us against 52.1 with 4 pieces); the rows are left in
// them for the attention that follows (nontemporal stores: 48.5 us).
constexpr int kAppendThreads = 256;

struct AppendArgs {
    const char* src[2];
    int64_t src_stride[2];      // bytes between tokens
    char* dst[2];
    const int64_t* slots;
    int64_t T;
    int64_t num_pages;
    int64_t page_stride;
    int64_t row_stride;         // of one head's rows inside a page
    int64_t head_stride;
    int32_t page_size;
    int32_t page_shift;         // log2(page_size), or -1
    uint32_t V;                 // pieces of a row
    uint32_t v_magic;           // ceil(2^32 / V) (0 for V = 1)
    uint32_t VH;                // pieces of a head
    uint32_t vh_magic;
    float scale[2];
    float inverse[2];           // 1 / scale, rounded
    unsigned long long* skipped;
};

__device__ inline uint32_t divide(uint32_t x, uint32_t magic) {
    return magic == 0 ? x : __umulhi(x, magic);
}

// Source elements of one 16-byte piece of the pool: the same bytes, or 16
// values to be rounded to e4m3 (nearest even, held at +-448; NaN stays NaN).
enum : int { kCopyBytes = 0, kFromBf16 = 1, kFromF16 = 2, kFromF32 = 3 };

template <int FROM>
struct Source {
    static constexpr int N = FROM == kCopyBytes ? 1 : (FROM == kFromF32 ? 4 : 2);   // 16-byte loads
    u32x4 x[N];
};

__device__ inline float held(float x) {
    // a comparison that NaN fails keeps it NaN
    return x > 448.0f ? 448.0f : (x < -448.0f ? -448.0f : x);
}

// x / scale, correctly rounded, from the rounded inverse: the quotient's
// remainder is exact, and corrects it (Markstein's theorem).  3 instructions for
// the dozen of a division, which bounded the kernel.
__device__ inline float quotient(float x, float scale, float inverse) {
    const float q = x * inverse;
    const float fine = __builtin_fmaf(__builtin_fmaf(-q, scale, x), inverse, q);
    return __builtin_fabsf(q) <= 1.0e6f ? fine : q;     // also no NaN from an infinity's remainder
}

template <int FROM>
__device__ inline u32x4 to_pool(const Source<FROM>& s, float scale, float inverse) {
    if constexpr (FROM == kCopyBytes) {
        return s.x[0];
    } else {
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (FROM == kFromF32) {
                const uint32_t w = s.x[i / 4][i % 4];   // a bit cast of the element itself reads element 0
                f[i] = __builtin_bit_cast(float, w);
            } else {
                const uint32_t w = s.x[i / 8][i % 8 / 2];
                const uint16_t h = static_cast<uint16_t>(i & 1 ? w >> 16 : w);
                if constexpr (FROM == kFromBf16)
                    f[i] = __builtin_bit_cast(float, static_cast<uint32_t>(h) << 16);
                else
                    f[i] = static_cast<float>(__builtin_bit_cast(_Float16, h));
            }
            f[i] = held(quotient(f[i], scale, inverse));
        }
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], w, true);
            r[i] = static_cast<uint32_t>(w);
        }
        return r;
    }
}

template <int FROM>
__global__ __launch_bounds__(kAppendThreads) void k_append(const AppendArgs A) {
    const int64_t piece0 = static_cast<int64_t>(blockIdx.x) * kAppendThreads;
    const int64_t row0 = piece0 / A.V;                  // rows: 2 t + (0 for K, 1 for V)
    const uint32_t f = static_cast<uint32_t>(piece0 - row0 * A.V) + threadIdx.x;
    const uint32_t rr = divide(f, A.v_magic);
    const uint32_t x = f - rr * A.V;
    const int64_t row = row0 + rr;
    const int64_t t = row >> 1;
    const int kv = static_cast<int>(row & 1);
    if (t >= A.T) return;
    const int64_t slot = A.slots[t];
    Source<FROM> src;
    const char* s = A.src[kv] + t * A.src_stride[kv] + static_cast<int64_t>(x) * (16 * Source<FROM>::N);
#pragma unroll
    for (int j = 0; j < Source<FROM>::N; ++j)
        src.x[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(s) + j);
    const int64_t page = A.page_shift >= 0 ? slot >> A.page_shift : slot / A.page_size;
    if (slot < 0 || page >= A.num_pages) {
        if (kv == 0 && x == 0 && A.skipped != nullptr) atomicAdd(A.skipped, 1ull);
        return;
    }
    const uint32_t h = divide(x, A.vh_magic);
    char* to = A.dst[kv] + page * A.page_stride + (slot - page * A.page_size) * A.row_stride +
               h * A.head_stride + (x - h * A.VH) * 16;
    *reinterpret_cast<u32x4*>(to) = to_pool<FROM>(src, A.scale[kv], A.inverse[kv]);
}

}  // namespace tables
}  // namespace kvx
