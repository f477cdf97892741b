// kvx_serve_host.hpp -- host side of include/kvx_serve.h: argument checks,
// tilings and launches.  Part of kvx.hip's translation unit, whose checks of
// layouts, pools, batches and tables it uses.
#pragma once

#include "kvx_attend.hpp"
#include "kvx_serve.h"
#include "kvx_tables.hpp"

#include <cmath>

namespace {

int32_t shift_of(int32_t page_size) {
    return (page_size & (page_size - 1)) == 0 ? __builtin_ctz(static_cast<uint32_t>(page_size)) : -1;
}

constexpr int32_t kMaxReqs = 1 << 24;          // requests (and groups) of a batch
constexpr int64_t kMaxQueries = 1 << 23;       // query tokens of an attention call, exclusive

bool positive(float x) { return std::isfinite(x) && x > 0.0f; }

// The debug checks copy tables to host vectors: a failed allocation is a
// status, and no exception passes the C entries.
template <class F>
kvx_status no_throw(F f) {
    try {
        return f();
    } catch (...) {
        return KVX_E_RANGE;
    }
}

// A launch's threads are counted in 32 bits.
bool launch_fits(int64_t grid, int threads) { return grid <= UINT32_MAX / threads; }

template <class Args>
kvx_status launch_one(const void* fn, int64_t grid, int threads, Args& a, hipStream_t stream) {
    if (grid <= 0) return KVX_OK;
    if (!launch_fits(grid, threads)) return KVX_E_RANGE;
    void* params[] = {&a};
    return hipLaunchKernel(fn, dim3(static_cast<uint32_t>(grid)), dim3(threads), params, 0, stream) ==
                   hipSuccess
               ? KVX_OK
               : KVX_E_HIP;
}

// Bytes of a buffer, to compare with another's (a count that passes the address
// space ends with it).
struct Extent {
    uintptr_t lo, hi;
    Extent(const void* p, int64_t count, int64_t size) : lo(reinterpret_cast<uintptr_t>(p)), hi(lo) {
        uintptr_t bytes = 0;
        if (p == nullptr || count <= 0) return;
        if (__builtin_mul_overflow(static_cast<uintptr_t>(count), static_cast<uintptr_t>(size), &bytes) ||
            __builtin_add_overflow(lo, bytes, &hi))
            hi = UINTPTR_MAX;
    }
    bool meets(const Extent& x) const { return std::max(lo, x.lo) < std::min(hi, x.hi); }
};

// ------------------------------------------------------------- building --

// The first workgroup writes lengths and offsets while others read theirs, and
// ids and slots are written window by window.
kvx_status check_build_overlap(int32_t n, const int32_t* have, const int32_t* add,
                               const kvx_table* held, const int32_t* free_ids, int64_t num_free,
                               const kvx_batch_tables* o) {
    const bool holds = have != nullptr && n > 0;
    const Extent in[] = {{have, n, 4},
                         {add, n, 4},
                         {holds ? held->pg_off : nullptr, n, 8},
                         {holds ? held->page_ids : nullptr, holds ? held->num_ids : 0, 4},
                         {free_ids, num_free, 4}};
    const Extent out[] = {{o->ctx_len, n, 4},
                          {o->tok_off, int64_t(n) + 1, 8},
                          {o->pg_off, int64_t(n) + 1, 8},
                          {o->page_ids, o->cap_ids, 4},
                          {o->slots, o->cap_tokens, 8},
                          {o->totals, 4, 8}};
    constexpr int N = sizeof(out) / sizeof(out[0]);
    for (int i = 0; i < N; ++i) {
        for (const Extent& x : in)
            if (out[i].meets(x)) return KVX_E_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return KVX_E_OVERLAP;
    }
    return KVX_OK;
}

kvx_status check_build(int32_t num_reqs, int32_t page_size, const int32_t* have,
                       const int32_t* add, const kvx_table* held, const int32_t* free_ids,
                       int64_t num_free, const kvx_batch_tables* o) {
    if (o == nullptr) return KVX_E_NULL;
    if (num_reqs < 0 || page_size < 1 || num_free < 0 || o->cap_ids < 0 || o->cap_tokens < 0)
        return KVX_E_SHAPE;
    if (num_reqs > kMaxReqs) return KVX_E_RANGE;
    if (num_free > 0 && free_ids == nullptr) return KVX_E_NULL;
    if (o->tok_off == nullptr || o->pg_off == nullptr) return KVX_E_NULL;
    if (num_reqs > 0 && (add == nullptr || o->ctx_len == nullptr)) return KVX_E_NULL;
    if ((o->cap_ids > 0 && o->page_ids == nullptr) || (o->cap_tokens > 0 && o->slots == nullptr))
        return KVX_E_NULL;
    if (have != nullptr && num_reqs > 0) {
        if (held == nullptr || held->pg_off == nullptr) return KVX_E_NULL;
        if (held->num_ids < 0) return KVX_E_SHAPE;
        if (held->num_ids > 0 && held->page_ids == nullptr) return KVX_E_NULL;
    }
    return KVX_OK;
}

// KVX_VALIDATE=1: lengths not negative, held lists inside their array, outputs large enough.
kvx_status validate_build(int32_t n, int32_t page, const int32_t* have, const int32_t* add,
                          const kvx_table* held, const kvx_batch_tables* o, hipStream_t stream) {
    if (n == 0) return KVX_OK;
    if (hipStreamSynchronize(stream) != hipSuccess) return KVX_E_HIP;
    std::vector<int32_t> h(static_cast<size_t>(n), 0), a;
    std::vector<int64_t> pg;
    KVX_TRY(to_host(add, n, &a));
    if (have != nullptr) {
        KVX_TRY(to_host(have, n, &h));
        KVX_TRY(to_host(held->pg_off, n, &pg));
    }
    int64_t tokens = 0, pages = 0;
    for (int32_t r = 0; r < n; ++r) {
        const size_t i = static_cast<size_t>(r);
        const int64_t hold = (static_cast<int64_t>(h[i]) + page - 1) / page;
        const bool bad = h[i] < 0 || a[i] < 0 || static_cast<int64_t>(h[i]) + a[i] > INT32_MAX ||
                         (hold > 0 && (pg[i] < 0 || pg[i] > held->num_ids - hold));
        if (bad) {
            std::fprintf(stderr, "kvx: KVX_VALIDATE: request %d's lengths or held pages; nothing "
                                 "enqueued\n", r);
            return KVX_E_SHAPE;
        }
        tokens += a[i];
        pages += (static_cast<int64_t>(h[i]) + a[i] + page - 1) / page;
    }
    return tokens > o->cap_tokens || pages > o->cap_ids ? KVX_E_SHAPE : KVX_OK;
}

// ------------------------------------------------------------ the layer --

// The planes, strides and checks that kvx_append and kvx_attend share.
struct LayerRef {
    Geom g;
    char* k;
    char* v;
    int64_t row_stride, page_stride, head_stride;
};

kvx_status check_layer(const kvx_layout* layout, int32_t layer, const kvx_pool* pool,
                       int32_t block_layout, LayerRef* ref) {
    KVX_TRY(check_layout(layout, &ref->g));
    if (layout->num_kv != 2) return KVX_E_UNSUPPORTED;
    if (layer < 0 || layer >= layout->num_layers) return KVX_E_SHAPE;
    if (block_layout != KVX_NHD && block_layout != KVX_HND) return KVX_E_SHAPE;
    const Geom& g = ref->g;
    if (pool == nullptr || pool->planes == nullptr) return KVX_E_NULL;
    // the two planes of the layer are all that the call touches
    kvx_pool two = *pool;
    two.planes = pool->planes + 2 * static_cast<int64_t>(layer);
    Geom g2 = g;
    g2.Q = 2;
    KVX_TRY(check_pool(&two, g2));
    ref->k = static_cast<char*>(two.planes[0]);
    ref->v = static_cast<char*>(two.planes[1]);
    ref->page_stride = page_stride_of(pool);
    if (block_layout == KVX_HND) {
        if (g.Db % 16 != 0) return KVX_E_ALIGN;
        ref->row_stride = g.Db;
        if (!mul_ok(pool->page_size, g.Db, &ref->head_stride)) return KVX_E_RANGE;
    } else {
        ref->row_stride = pool->slot_stride;
        ref->head_stride = g.Db;
    }
    return KVX_OK;
}

// KVX_VALIDATE=1: no slot of the pool is written twice, and no row of k or v
// (`row` bytes) lies in one that is written.
kvx_status validate_append(const LayerRef& ref, int32_t block_layout, const kvx_pool* pool,
                           const int64_t* slots, const kvx_rows* rows, int64_t row,
                           hipStream_t stream) {
    if (hipStreamSynchronize(stream) != hipSuccess) return KVX_E_HIP;
    std::vector<int64_t> at;
    KVX_TRY(to_host(slots, rows->num_tokens, &at));
    auto skipped = [&](int64_t x) { return x < 0 || x / pool->page_size >= pool->num_pages; };
    std::vector<int64_t> s = at;
    s.erase(std::remove_if(s.begin(), s.end(), skipped), s.end());
    std::sort(s.begin(), s.end());
    const auto twice = std::adjacent_find(s.begin(), s.end());
    if (twice != s.end()) {
        std::fprintf(stderr, "kvx: KVX_VALIDATE: append: slot %lld twice; nothing enqueued\n",
                     static_cast<long long>(*twice));
        return KVX_E_DUPLICATE;
    }
    const int64_t runs = block_layout == KVX_HND ? ref.g.H : 1;     // a head-major row is a run per head
    std::vector<Span> written, read;
    for (int64_t t = 0; t < rows->num_tokens; ++t) {
        const int64_t x = at[static_cast<size_t>(t)];
        if (skipped(x)) continue;
        const uint64_t off = static_cast<uint64_t>(x / pool->page_size * ref.page_stride +
                                                   x % pool->page_size * ref.row_stride);
        for (const char* plane : {ref.k, ref.v})
            for (int64_t h = 0; h < runs; ++h) {
                const uint64_t lo = reinterpret_cast<uint64_t>(plane) + off +
                                    static_cast<uint64_t>(h * ref.head_stride);
                written.push_back(Span{lo, lo + static_cast<uint64_t>(ref.g.R / runs), t});
            }
        const uint64_t k = reinterpret_cast<uint64_t>(rows->k) + static_cast<uint64_t>(t * rows->k_stride);
        const uint64_t v = reinterpret_cast<uint64_t>(rows->v) + static_cast<uint64_t>(t * rows->v_stride);
        read.push_back(Span{k, k + static_cast<uint64_t>(row), t});
        read.push_back(Span{v, v + static_cast<uint64_t>(row), t});
    }
    int64_t bad = 0;
    const kvx_status st = spans_disjoint(&written, &read, &bad);
    if (st != KVX_OK)
        std::fprintf(stderr, "kvx: KVX_VALIDATE: append: a row is %s (token %lld); nothing enqueued\n",
                     st == KVX_E_OVERLAP ? "read and written" : "written twice",
                     static_cast<long long>(bad));
    return st;
}

// ------------------------------------------------------------ attention --

namespace at = kvx::attend;

constexpr int64_t kAttendGrid = 256;    // one workgroup per compute unit of an MI355X
constexpr int64_t kJoinPlaces = 2048;   // waves of a join that shares rows among waves

// The average query rows per kv head of a batch's contexts (and those of its
// prefixes) decide their tiles, one kind for all: wide ones from kWideRows on.
// The host has no lengths but total_tokens, so rows that a padded batch does not
// use count too, and in a batch that mixes prompts with single tokens one of the
// two runs in the other's tiles (63 tokens from e4m3 beside a prompt of 2048: 226
// us, apart 60 + 87; 255 beside a chunk of 512: 253, apart 209 + 56).  Contexts
// all alike, 64 of 2048 keys, thin against wide: 8 kv heads of 128 dims with 16 /
// 32 / 64 / 128 rows 123 : 130, 142 : 132, 202 : 134, 384 : 149 us; with 64 dims
// 66 : 85, 81 : 86, 125 : 87, 230 : 89; from e4m3 73 : 132, 94 : 133, 143 : 135,
// 265 : 139. Above 128 dims of 16 bits K and V of a step ahead and the
// accumulators pass a wave's registers, and wide tiles win at any number of rows
// (256 dims, 4 kv heads: 1 row 152 : 110, 16 rows 159 : 112; 4 contexts 47 : 26;
// 512 of 300 keys 185 : 157): these have no thin ones.
constexpr int64_t kWideRows = 64;

struct AttendShape {
    int DP;
    int32_t G;
    bool pre_wide, own_wide;
    int32_t wide_rows;
    int32_t slot_rows;
    int64_t placed, plan, splits, slot_ml, slot_o, row_ml, row_o, bytes;    // offsets into the workspace
};

kvx_status attend_shape(const kvx_layout* layout, const Geom& g, int32_t num_reqs,
                        int32_t num_groups, int64_t tokens, int32_t q_heads, AttendShape* s) {
    if (layout->num_kv != 2 || layout->dtype == KVX_F32 || layout->head_dim > 256)
        return KVX_E_UNSUPPORTED;
    if (g.Db % 16 != 0) return KVX_E_ALIGN;
    if (num_reqs < 0 || num_groups < 0 || tokens < 0 || q_heads < 1 || q_heads % g.H != 0)
        return KVX_E_SHAPE;
    if (q_heads / g.H > 128 || tokens >= kMaxQueries || num_reqs > kMaxReqs || num_groups > kMaxReqs)
        return KVX_E_RANGE;
    const int32_t D = layout->head_dim;
    s->DP = D <= 64 ? 64 : (D <= 128 ? 128 : 256);
    s->G = q_heads / g.H;
    const int64_t rows = tokens * s->G;
    const bool all_wide = s->DP > 128 && layout->dtype != KVX_FP8;
    s->own_wide = num_reqs > 0 && (all_wide || rows / num_reqs >= kWideRows);
    s->pre_wide = num_groups > 0 && (all_wide || rows / num_groups >= kWideRows);
    s->wide_rows = s->DP <= 128 ? 256 : 128;
    // of the larger tile whichever this batch takes, so that a smaller batch needs no more
    s->slot_rows = std::max(s->wide_rows, at::kWaves * at::kThinRows);
    int64_t end = 0;
    auto take = [&](int64_t count, int64_t size) {
        const int64_t at0 = end;
        int64_t b = 0;
        if (end < 0 || !mul_ok(count, size, &b) || b > (int64_t(1) << 60)) { end = -1; return at0; }
        end += (b + 255) / 256 * 256;
        return at0;
    };
    s->placed = take(static_cast<int64_t>(num_reqs) + num_groups, sizeof(at::Placed));
    s->plan = take(6, 8);
    s->splits = take(kAttendGrid, sizeof(at::Split));
    s->slot_ml = take(2 * kAttendGrid * s->slot_rows, 8);
    s->slot_o = take(2 * kAttendGrid * s->slot_rows, 4 * static_cast<int64_t>(D));
    int64_t out_rows = 0;
    if (!mul_ok(tokens, q_heads, &out_rows)) return KVX_E_RANGE;
    if (num_groups == 0) out_rows = 0;
    s->row_ml = take(2 * out_rows, 8);
    s->row_o = take(2 * out_rows, 4 * static_cast<int64_t>(D));
    if (end < 0) return KVX_E_RANGE;
    s->bytes = end;
    return KVX_OK;
}

struct AttendKernels {
    const void *main, *join, *join_shared, *join_items;
};

template <class T, bool FP8, int DP>
AttendKernels attend_kernels(int lines) {
    const void* main;
    if constexpr (DP > 128 && !FP8)
        main = reinterpret_cast<const void*>(&at::k_attend<T, FP8, DP, 2>);
    else
        main = lines == 1 ? reinterpret_cast<const void*>(&at::k_attend<T, FP8, DP, 1>)
                          : reinterpret_cast<const void*>(&at::k_attend<T, FP8, DP, 3>);
    return {main, reinterpret_cast<const void*>(&at::k_attend_join<T, DP, false>),
            reinterpret_cast<const void*>(&at::k_attend_join<T, DP, true>),
            reinterpret_cast<const void*>(&at::k_attend_join_items<T, DP>)};
}

template <class T, bool FP8>
AttendKernels attend_kernels(int DP, int lines) {
    return DP == 64    ? attend_kernels<T, FP8, 64>(lines)
           : DP == 128 ? attend_kernels<T, FP8, 128>(lines)
                       : attend_kernels<T, FP8, 256>(lines);
}

// n rows of `len` bytes, `stride` apart.
struct StridedRows {
    const void* at;
    int64_t stride, len, n;
};

// Whether a row of `a` shares a byte with a row of `b`.  q and out may be slices
// of one fused buffer, whose spans overlap while their rows do not.
bool rows_meet(const StridedRows& a, const StridedRows& b) {
    if (a.at == nullptr || b.at == nullptr) return false;
    const Extent ea(a.at, (a.n - 1) * a.stride + a.len, 1), eb(b.at, (b.n - 1) * b.stride + b.len, 1);
    if (!ea.meets(eb)) return false;
    // rows i of a and j of b, k = i - j, of one stride s meet if and only if
    // -a.len < d + k s < b.len, d = a - b: the smallest k for the left side
    // decides.  With other strides, one row of b after the other.
    const int64_t d0 = static_cast<int64_t>(ea.lo - eb.lo), s = a.stride;
    const bool alike = a.stride == b.stride;
    for (int64_t j = 0; j < (alike ? 1 : b.n); ++j) {
        const int64_t d = d0 - j * b.stride, x = -a.len - d;
        int64_t k = (x >= 0 ? x / s : -((-x + s - 1) / s)) + 1;
        k = std::max(k, alike ? 1 - b.n : int64_t(0));
        if (k < a.n && d + k * s < b.len) return true;
    }
    return false;
}

kvx_status validate_attend(const kvx_reqs* reqs, const int32_t* ctx, const kvx_prefix* prefix,
                           hipStream_t stream) {
    if (hipStreamSynchronize(stream) != hipSuccess) return KVX_E_HIP;
    std::vector<int64_t> off;
    std::vector<int32_t> len;
    KVX_TRY(to_host(reqs->tok_off, static_cast<int64_t>(reqs->num_reqs) + 1, &off));
    const kvx_reqs hr{reqs->num_reqs, std::min(off.back(), reqs->total_tokens), off.data()};
    kvx_status s = check_tok_off(&hr);
    KVX_TRY(to_host(ctx, reqs->num_reqs, &len));
    for (int32_t x : len)
        if (x < 0 || x > at::kMaxKeys) s = KVX_E_SHAPE;
    if (prefix != nullptr && prefix->num_groups > 0) {
        KVX_TRY(to_host(prefix->grp_off, static_cast<int64_t>(prefix->num_groups) + 1, &off));
        const kvx_reqs hg{prefix->num_groups, reqs->num_reqs, off.data()};
        if (s == KVX_OK) s = check_tok_off(&hg);
        KVX_TRY(to_host(prefix->len, prefix->num_groups, &len));
        for (int32_t x : len)
            if (x < 0 || x > at::kMaxKeys) s = KVX_E_SHAPE;
    }
    if (s != KVX_OK)
        std::fprintf(stderr, "kvx: KVX_VALIDATE: attend: %s; nothing enqueued\n", kvx_status_str(s));
    return s;
}

}  // namespace

extern "C" {

kvx_status kvx_build_tables(int32_t num_reqs, int32_t page_size, const int32_t* have_len,
                            const int32_t* add_len, const kvx_table* held,
                            const int32_t* free_ids, int64_t num_free,
                            const kvx_batch_tables* out, hipStream_t stream) {
    namespace tb = kvx::tables;
    KVX_TRY(check_build(num_reqs, page_size, have_len, add_len, held, free_ids, num_free, out));
    tb::BuildArgs a;
    std::memset(&a, 0, sizeof(a));
    a.have = num_reqs > 0 ? have_len : nullptr;
    a.add = add_len;
    if (a.have != nullptr) {
        a.held_off = held->pg_off;
        a.held_ids = held->page_ids;
        a.num_held = held->num_ids;
    }
    a.free_ids = free_ids;
    a.num_free = num_free;
    a.num_reqs = num_reqs;
    a.page_size = page_size;
    a.page_shift = shift_of(page_size);
    a.ctx = out->ctx_len;
    a.tok_off = out->tok_off;
    a.pg_off = out->pg_off;
    a.ids = out->page_ids;
    a.cap_ids = out->cap_ids;
    a.slots = out->slots;
    a.cap_tokens = out->cap_tokens;
    a.totals = out->totals;
    auto grid_of = [&](int64_t slot_run, int64_t id_run) {
        const int64_t s = slot_run * tb::kBuildThreads, i = id_run * tb::kBuildThreads;
        return std::max<int64_t>(1, std::max(out->cap_tokens / s + (out->cap_tokens % s != 0),
                                             out->cap_ids / i + (out->cap_ids % i != 0)));
    };
    const bool few = num_reqs <= tb::kFewRequests;
    int64_t grid = grid_of(1, 1);
    const void* fn = few ? reinterpret_cast<const void*>(&tb::k_build_tables<1, 1, 1>)
                         : reinterpret_cast<const void*>(&tb::k_build_tables<1, 1, tb::kManyPerThread>);
    if (grid > tb::kShortGrid) {
        constexpr int S = tb::kLongSlotRun, I = tb::kLongIdRun;
        grid = grid_of(S, I);
        fn = few ? reinterpret_cast<const void*>(&tb::k_build_tables<S, I, 1>)
                 : reinterpret_cast<const void*>(&tb::k_build_tables<S, I, tb::kManyPerThread>);
    }
    if (!launch_fits(grid, tb::kBuildThreads)) return KVX_E_RANGE;
    KVX_TRY(check_build_overlap(num_reqs, have_len, add_len, held, free_ids, num_free, out));
    if (validate_enabled())
        KVX_TRY(no_throw([&] {
            return validate_build(num_reqs, page_size, have_len, add_len, held, out, stream);
        }));
    if (log_enabled())
        std::fprintf(stderr, "kvx: build_tables reqs=%d page=%d grid=%lld\n", num_reqs, page_size,
                     static_cast<long long>(grid));
    return launch_one(fn, grid, tb::kBuildThreads, a, stream);
}

kvx_status kvx_append(const kvx_layout* layout, int32_t layer, const kvx_pool* pool,
                      int32_t block_layout, const int64_t* slots, const kvx_rows* rows,
                      unsigned long long* skipped, hipStream_t stream) {
    namespace tb = kvx::tables;
    LayerRef ref;
    KVX_TRY(check_layer(layout, layer, pool, block_layout, &ref));
    const Geom& g = ref.g;
    if (rows == nullptr) return KVX_E_NULL;
    const int eb = elem_bytes(rows->dtype);
    if (eb == 0) return KVX_E_DTYPE;
    if (rows->num_tokens < 0) return KVX_E_SHAPE;
    if (rows->num_tokens >= (int64_t(1) << 31)) return KVX_E_RANGE;
    const bool copies = rows->dtype == layout->dtype;
    if (!copies && layout->dtype != KVX_FP8) return KVX_E_UNSUPPORTED;
    if (!positive(rows->k_scale) || !positive(rows->v_scale)) return KVX_E_SHAPE;
    // inside these the kernel's quotients by a rounded inverse are exact: no
    // remainder of a value that e4m3 holds underflows
    auto far = [](float x) { return x < 0x1p-64f || x > 0x1p64f; };
    if (far(rows->k_scale) || far(rows->v_scale)) return KVX_E_RANGE;
    if (copies && (rows->k_scale != 1.0f || rows->v_scale != 1.0f)) return KVX_E_UNSUPPORTED;
    if (rows->num_tokens == 0) return KVX_OK;
    if (rows->k == nullptr || rows->v == nullptr || slots == nullptr) return KVX_E_NULL;
    const int64_t row = static_cast<int64_t>(layout->kv_heads) * layout->head_dim * eb;
    if (rows->k_stride < row || rows->v_stride < row) return KVX_E_SHAPE;
    if (!aligned16(rows->k) || !aligned16(rows->v) || rows->k_stride % 16 != 0 ||
        rows->v_stride % 16 != 0)
        return KVX_E_ALIGN;
    int64_t span = 0;
    if (!mul_ok(rows->num_tokens, std::max(rows->k_stride, rows->v_stride), &span))
        return KVX_E_RANGE;
    if (validate_enabled())
        KVX_TRY(no_throw([&] {
            return validate_append(ref, block_layout, pool, slots, rows, row, stream);
        }));
    tb::AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    a.src[0] = static_cast<const char*>(rows->k);
    a.src[1] = static_cast<const char*>(rows->v);
    a.src_stride[0] = rows->k_stride;
    a.src_stride[1] = rows->v_stride;
    a.dst[0] = ref.k;
    a.dst[1] = ref.v;
    a.slots = slots;
    a.T = rows->num_tokens;
    a.num_pages = pool->num_pages;
    a.page_stride = ref.page_stride;
    a.row_stride = ref.row_stride;
    a.page_size = pool->page_size;
    a.page_shift = shift_of(pool->page_size);
    a.V = static_cast<uint32_t>(g.R / 16);
    // an NHD row is one run; an HND row is a run per head
    a.VH = block_layout == KVX_HND ? static_cast<uint32_t>(g.Db / 16) : a.V;
    a.head_stride = block_layout == KVX_HND ? ref.head_stride : 0;
    auto magic = [](uint32_t v) {
        return v == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + v - 1) / v);
    };
    a.v_magic = magic(a.V);
    a.vh_magic = magic(a.VH);
    a.scale[0] = rows->k_scale;
    a.scale[1] = rows->v_scale;
    a.inverse[0] = 1.0f / rows->k_scale;
    a.inverse[1] = 1.0f / rows->v_scale;
    a.skipped = skipped;
    const int64_t per = tb::kAppendThreads;
    const int64_t grid = (rows->num_tokens * 2 * a.V + per - 1) / per;
    const void* fn = reinterpret_cast<const void*>(&tb::k_append<tb::kCopyBytes>);
    if (!copies)
        fn = rows->dtype == KVX_BF16  ? reinterpret_cast<const void*>(&tb::k_append<tb::kFromBf16>)
             : rows->dtype == KVX_F16 ? reinterpret_cast<const void*>(&tb::k_append<tb::kFromF16>)
                                      : reinterpret_cast<const void*>(&tb::k_append<tb::kFromF32>);
    if (log_enabled())
        std::fprintf(stderr, "kvx: append tokens=%lld row=%lld grid=%lld\n",
                     static_cast<long long>(a.T), static_cast<long long>(g.R),
                     static_cast<long long>(grid));
    return launch_one(fn, grid, tb::kAppendThreads, a, stream);
}

kvx_status kvx_attend_workspace(const kvx_layout* layout, int32_t num_reqs, int32_t num_groups,
                                int64_t total_tokens, int32_t q_heads, int64_t* bytes) {
    Geom g;
    if (bytes == nullptr) return KVX_E_NULL;
    KVX_TRY(check_layout(layout, &g));
    AttendShape s;
    KVX_TRY(attend_shape(layout, g, num_reqs, num_groups, total_tokens, q_heads, &s));
    *bytes = s.bytes;
    return KVX_OK;
}

kvx_status kvx_attend(const kvx_layout* layout, int32_t layer, const kvx_pool* pool,
                      int32_t block_layout, const kvx_reqs* reqs, const int32_t* ctx_len,
                      const kvx_table* table, const kvx_prefix* prefix,
                      const kvx_attention* attention, unsigned long long* skipped,
                      hipStream_t stream) {
    LayerRef ref;
    KVX_TRY(check_layer(layout, layer, pool, block_layout, &ref));
    const Geom& g = ref.g;
    KVX_TRY(check_reqs(reqs));
    if (attention == nullptr) return KVX_E_NULL;
    const kvx_attention& x = *attention;
    if ((x.flags & ~KVX_ATTEND_CAUSAL) != 0) return KVX_E_UNSUPPORTED;
    if (x.dtype != KVX_F16 && x.dtype != KVX_BF16)
        return elem_bytes(x.dtype) == 0 ? KVX_E_DTYPE : KVX_E_UNSUPPORTED;
    if (layout->dtype != x.dtype && layout->dtype != KVX_FP8) return KVX_E_UNSUPPORTED;
    const int32_t ng = prefix != nullptr ? prefix->num_groups : 0;
    AttendShape s;
    KVX_TRY(attend_shape(layout, g, reqs->num_reqs, ng, reqs->total_tokens, x.q_heads, &s));
    if (!positive(x.scale) || !positive(x.k_scale) || !positive(x.v_scale)) return KVX_E_SHAPE;
    const float scale = x.scale * x.k_scale * 1.4426950408889634f;
    if (!positive(scale)) return KVX_E_RANGE;
    KVX_TRY(check_table(table, reqs));
    if (reqs->num_reqs > 0 && ctx_len == nullptr) return KVX_E_NULL;
    if (ng > 0) {
        const kvx_reqs groups{ng, reqs->num_reqs, prefix->grp_off};
        KVX_TRY(check_reqs(&groups));
        KVX_TRY(check_table(&prefix->table, &groups));
        if (prefix->len == nullptr) return KVX_E_NULL;
    }
    if (reqs->num_reqs == 0 || reqs->total_tokens == 0) return KVX_OK;
    KVX_TRY(check_source_nonempty(pool, reqs));
    if (x.q == nullptr || x.out == nullptr || x.workspace == nullptr) return KVX_E_NULL;
    const int64_t row = static_cast<int64_t>(x.q_heads) * layout->head_dim * 2;
    int64_t span = 0;
    if (x.q_stride < row || x.out_stride < row) return KVX_E_SHAPE;
    if (!mul_ok(reqs->total_tokens, std::max(x.q_stride, x.out_stride), &span)) return KVX_E_RANGE;
    if (!aligned16(x.q) || !aligned16(x.out) || x.q_stride % 16 != 0 || x.out_stride % 16 != 0 ||
        (reinterpret_cast<uintptr_t>(x.workspace) & 255u) != 0 ||
        (reinterpret_cast<uintptr_t>(x.lse) & 3u) != 0)
        return KVX_E_ALIGN;
    if (x.workspace_bytes < s.bytes) return KVX_E_SHAPE;
    const int64_t T = reqs->total_tokens, lse_bytes = T * x.q_heads * 4;    // inside T * row
    const StridedRows buffers[] = {{x.q, x.q_stride, row, T},
                                   {x.out, x.out_stride, row, T},
                                   {x.lse, lse_bytes, lse_bytes, 1},
                                   {x.workspace, s.bytes, s.bytes, 1}};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (rows_meet(buffers[i], buffers[j])) return KVX_E_OVERLAP;
    if (validate_enabled())
        KVX_TRY(no_throw([&] { return validate_attend(reqs, ctx_len, prefix, stream); }));

    at::Args a;
    std::memset(&a, 0, sizeof(a));
    a.k = ref.k;
    a.v = ref.v;
    a.row_stride = ref.row_stride;
    a.page_stride = ref.page_stride;
    a.head_stride = ref.head_stride;
    a.num_pages = pool->num_pages;
    a.page_size = pool->page_size;
    a.page_shift = shift_of(pool->page_size);
    a.tok_off = reqs->tok_off;
    a.ctx = ctx_len;
    a.own = at::Lists{table->pg_off, table->page_ids, table->num_ids};
    if (ng > 0) {
        a.grp_off = prefix->grp_off;
        a.plen = prefix->len;
        a.pre = at::Lists{prefix->table.pg_off, prefix->table.page_ids, prefix->table.num_ids};
    }
    a.q = static_cast<const char*>(x.q);
    a.out = static_cast<char*>(x.out);
    a.lse = x.lse;
    a.q_stride = x.q_stride;
    a.out_stride = x.out_stride;
    a.skipped = skipped;
    a.T = static_cast<int32_t>(reqs->total_tokens);
    a.num_reqs = reqs->num_reqs;
    a.num_groups = ng;
    a.H = g.H;
    a.G = s.G;
    a.D = layout->head_dim;
    a.causal = (x.flags & KVX_ATTEND_CAUSAL) != 0;
    a.scale = scale;
    a.v_scale = x.v_scale;
    // thin tiles: a kv head's query heads in as few parts of at most 16 as
    // there can be, the thin heads in as few sets of at most 8 waves
    a.parts = (s.G + at::kThinRows - 1) / at::kThinRows;
    a.gv = (s.G + a.parts - 1) / a.parts;
    const int32_t heads = g.H * a.parts;
    a.sets = (heads + at::kWaves - 1) / at::kWaves;
    a.hs = (heads + a.sets - 1) / a.sets;
    a.sets = (heads + a.hs - 1) / a.hs;
    a.kp = at::kWaves / a.hs;
    a.thin_tokens = at::kThinRows / a.gv;
    a.wide_tokens = s.wide_rows / s.G;
    a.pre_wide = s.pre_wide;
    a.own_wide = s.own_wide;
    // The fewest units of a piece, and the units that an item's fixed time
    // (queries, first loads, stores) counts for.  Shorter pieces spread a small
    // batch over more workgroups and leave more to join: with 2^5 / 2^6 / 2^7
    // units 4 contexts of 300 keys take 19.9 / 21.4 / 22.5 us, 4 of 2048 keys
    // 28.1 / 22.9 / 26.5, 64 of 64 keys 19.1 / 20.5 / 16.5, one of 8192 keys 33.1 /
    // 26.4 / 28.3.  Items of 40 to 100 (thin) and 320 to 600 units (wide) are
    // within 3% of each other on ragged batches; without them the workgroups
    // with many short items end last.
    a.thin_min_log2 = 6;
    a.wide_min_log2 = 8;
    a.thin_item = 64;
    a.wide_item = 450;
    // a compute unit's time for a wide key (its products, 2350 a ns) over that
    // for a thin key (its bytes, 26 a ns): rates of the two loops alone
    const double wide_ns = 4.0 * s.wide_rows * s.DP / 2350.0;
    const double thin_ns = 2.0 * a.hs * g.Db / a.parts / 26.0;
    a.wide_weight = static_cast<float>(wide_ns / thin_ns);
    char* ws = static_cast<char*>(x.workspace);
    a.placed = reinterpret_cast<at::Placed*>(ws + s.placed);
    a.plan = reinterpret_cast<int64_t*>(ws + s.plan);
    a.splits = reinterpret_cast<at::Split*>(ws + s.splits);
    a.slot_ml = reinterpret_cast<float*>(ws + s.slot_ml);
    a.slot_o = reinterpret_cast<float*>(ws + s.slot_o);
    a.row_ml = reinterpret_cast<float*>(ws + s.row_ml);
    a.row_o = reinterpret_cast<float*>(ws + s.row_o);
    a.slot_rows = s.slot_rows;

    const int lines = s.own_wide || s.pre_wide ? 3 : 1;
    const bool fp8 = layout->dtype == KVX_FP8;
    const AttendKernels k = x.dtype == KVX_BF16
                                ? (fp8 ? attend_kernels<__bf16, true>(s.DP, lines)
                                       : attend_kernels<__bf16, false>(s.DP, lines))
                                : (fp8 ? attend_kernels<_Float16, true>(s.DP, lines)
                                       : attend_kernels<_Float16, false>(s.DP, lines));
    if (log_enabled())
        std::fprintf(stderr,
                     "kvx: attend reqs=%d groups=%d tokens=%lld heads=%d/%d dim=%d prefix=%s own=%s\n",
                     a.num_reqs, ng, static_cast<long long>(a.T), x.q_heads, g.H, a.D,
                     ng == 0 ? "none" : (s.pre_wide ? "wide" : "thin"), s.own_wide ? "wide" : "thin");
    KVX_TRY(launch_one(k.main, kAttendGrid, at::kThreads, a, stream));
    if (ng > 0) {
        const int32_t per_head = (a.gv + 256 / s.DP - 1) / (256 / s.DP);
        const int32_t units = heads * per_head;
        // waves that share a row's pieces, so that a few rows' many pieces are
        // not one wave's each (4 requests behind a prefix of 4096 tokens 50 -> 28
        // us); with many rows the waves are better spent on those (64 requests
        // in 8 groups 36 us; 41 with 4 waves a row)
        int32_t ways = at::kJoinWaves;
        while (ways > 1 && static_cast<int64_t>(a.T) * units * ways > kJoinPlaces) ways /= 2;
        const uint32_t deep = (units * ways + at::kJoinWaves - 1) / at::kJoinWaves;
        void* join_params[] = {&a, &ways};
        return hipLaunchKernel(ways > 1 ? k.join_shared : k.join, dim3(static_cast<uint32_t>(a.T), deep), dim3(64 * at::kJoinWaves),
                               join_params, 0, stream) == hipSuccess
                   ? KVX_OK
                   : KVX_E_HIP;
    }
    int32_t pieces = static_cast<int32_t>(kAttendGrid);
    const int64_t grid = pieces * at::kJoinParts +
                         (a.num_reqs + 64 * at::kJoinWaves - 1) / (64 * at::kJoinWaves);
    void* params[] = {&a, &pieces};
    return hipLaunchKernel(k.join_items, dim3(static_cast<uint32_t>(grid)), dim3(64 * at::kJoinWaves), params,
                           0, stream) == hipSuccess
               ? KVX_OK
               : KVX_E_HIP;
}

}  // extern "C"
