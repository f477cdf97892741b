/*
 * kvx_serve.h -- the serving step around a paged pool, in libkvx.so beside the
 * calls of kvx.h: page tables and slot maps from request lengths, new K/V rows
 * written into the pool, and attention over the pool for requests that share
 * prefixes.  A step of a decoder is
 *
 *   kvx_build_tables   lengths -> token offsets, page table, slots   (once)
 *   kvx_append         a layer's new K and V rows -> the pool        (per layer)
 *   kvx_attend         queries against prefix and own context        (per layer)
 *
 * The conventions of kvx.h hold: layouts, pools, pages, tables and request
 * batches are its structs; every call checks its arguments on the host,
 * enqueues its kernels on `stream` and returns; nothing is allocated and no
 * state is kept; an error enqueues nothing.  All lengths, offsets and ids stay
 * on the device, so a step can be captured once and replayed while they
 * change.  The calls record kernel launches only.  With KVX_VALIDATE=1 each
 * call first checks its device tables on the host, as stated below.  Host
 * structs are read only during the call.  Launches go to the current device,
 * which has to be the stream's and the buffers'.
 */
#ifndef KVX_SERVE_H
#define KVX_SERVE_H

#include "kvx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Outputs of kvx_build_tables, all DEVICE.  Entries past the counts that the
 * batch needs keep their prior contents (a replayed step whose batches shrink
 * fills slots with -1 first, and kvx_append skips the rows behind the last). */
typedef struct kvx_batch_tables {
    int32_t* ctx_len;       /* [num_reqs] have + add */
    int64_t* tok_off;       /* [num_reqs + 1] offsets of the new tokens (kvx_reqs) */
    int64_t* pg_off;        /* [num_reqs + 1] offsets into page_ids (kvx_table) */
    int32_t* page_ids;      /* [cap_ids] every page of every request */
    int64_t cap_ids;        /* >= 0; ids past it are not written */
    int64_t* slots;         /* [cap_tokens] slot of each new token */
    int64_t cap_tokens;     /* >= 0; slots past it are not written */
    int64_t* totals;        /* NULL or [4]: new tokens, pages, pages taken from the
                             * free list, pages the free list was short of */
} kvx_batch_tables;

/* Tables from lengths.  Request r holds have_len[r] tokens (NULL: none) in the
 * pages of `held` (their ids start at held->page_ids[held->pg_off[r]]) and gets
 * add_len[r] more.  Its new table is its ceil(have / page_size) held pages
 * followed by the new ones it needs, which are taken from free_ids in order,
 * request by request, from free_ids[0] on.  New token i of request r gets
 *   slots[tok_off[r] + i] = page * page_size + t % page_size,  t = have + i,
 * in page t / page_size of the new table.  A page past the end of free_ids,
 * or a held one outside held->page_ids, is written as -1, and a token in a page
 * with a negative id gets slot -1: kvx's calls skip such rows.  Negative
 * lengths count as 0, and a request's total stops at 2^31 - 1 tokens.  At most
 * 2^24 requests (KVX_E_RANGE).  No output may overlap an input (the lengths and
 * the held table are read while the new ones are written) or another output:
 * KVX_E_OVERLAP, by the arrays' addresses and sizes.  One launch. */
kvx_status kvx_build_tables(int32_t num_reqs, int32_t page_size, const int32_t* have_len,
                            const int32_t* add_len, const kvx_table* held,
                            const int32_t* free_ids, int64_t num_free,
                            const kvx_batch_tables* out, hipStream_t stream);

/* New rows of one layer.  k and v are DEVICE [num_tokens][kv_heads][head_dim]
 * tensors of `dtype` (a kvx_dtype), dense in their last two dimensions, their
 * tokens k_stride and v_stride bytes apart (multiples of 16; a row of a fused
 * projection's output is fine).  Row t goes to slot slots[t] of the layer's K
 * and V planes, in NHD or HND blocks (kvx_block_layout).  The rows are copied
 * bit by bit where dtype is the pool's; a KVX_FP8 pool also takes f16, bf16 and
 * f32 rows, which it holds as e4m3 (OCP, nearest even) of x / k_scale and
 * x / v_scale, values past +-448 held at +-448 and NaN kept.  A KVX_FP4 pool
 * takes f16, bf16 and f32 rows: each block of 32 dims is held under the smallest
 * 2^e that leaves its largest |x / scale| (32 bits) at most 7 * 2^e, e inside
 * -23 .. 13, its numbers rounded to the nearest of x / scale / 2^e (ties to the
 * even code, past 6 to 6, so that an infinity is held as 6), and a block with a
 * NaN as 32 of them; every held value is exact in f16, bf16 and f32, and a row's
 * padding keeps its contents.  (Other pairs: KVX_E_UNSUPPORTED.)  Scales are
 * finite, positive and from 2^-64 to 2^64 (KVX_E_RANGE), and 1 is required where
 * nothing is rounded.  A slot outside the
 * pool is skipped and counted once in *skipped (if not NULL).  Distinct tokens
 * have distinct slots, and no row of k or v lies in a slot that the call writes
 * (a page may be copied to another); both are unchecked, and KVX_VALIDATE=1
 * returns KVX_E_DUPLICATE or KVX_E_OVERLAP.  The layout has num_kv = 2.  One
 * launch. */
typedef struct kvx_rows {
    const void* k;
    const void* v;
    int64_t k_stride;
    int64_t v_stride;
    int64_t num_tokens;
    int32_t dtype;
    float k_scale;
    float v_scale;
} kvx_rows;

kvx_status kvx_append(const kvx_layout* layout, int32_t layer, const kvx_pool* pool,
                      int32_t block_layout, const int64_t* slots, const kvx_rows* rows,
                      unsigned long long* skipped, hipStream_t stream);

/* Shared prefixes: group g is requests [grp_off[g], grp_off[g + 1]), all of
 * whose tokens see the first len[g] tokens of table entry g.  grp_off is a
 * DEVICE array of num_groups + 1 int64 values with grp_off[0] = 0,
 * non-decreasing, grp_off[num_groups] = num_reqs; a group without a prefix has
 * length 0. */
typedef struct kvx_prefix {
    int32_t num_groups;
    const int64_t* grp_off;
    const int32_t* len;     /* DEVICE [num_groups] */
    kvx_table table;        /* pg_off has num_groups + 1 entries */
} kvx_prefix;

#define KVX_ATTEND_CAUSAL 1u

typedef struct kvx_attention {
    const void* q;          /* DEVICE [total_tokens][q_heads][head_dim] */
    void* out;              /* DEVICE, of the same shape and type */
    float* lse;             /* NULL or DEVICE [total_tokens][q_heads] */
    int64_t q_stride;       /* bytes between tokens: multiples of 16, at least a row */
    int64_t out_stride;
    int32_t q_heads;        /* a multiple of kv_heads, at most 128 per kv head */
    int32_t dtype;          /* KVX_F16 or KVX_BF16: of q and out */
    float scale;            /* of q.k; finite and positive */
    float k_scale;          /* the pool's values times this are K (1 for none) */
    float v_scale;
    uint32_t flags;         /* 0 or KVX_ATTEND_CAUSAL */
    void* workspace;        /* DEVICE, 256-byte aligned */
    int64_t workspace_bytes;
} kvx_attention;

/* Attention of a batch's query tokens over one layer of a paged pool.
 *
 * Query token i of request r (reqs: its n tokens are [tok_off[r],
 * tok_off[r + 1])) sees all keys of its group's prefix and, of the first
 * c = ctx_len[r] tokens of table entry r, those with index at most c - n + i
 * under KVX_ATTEND_CAUSAL (its own tokens are the context's last n), all of
 * them otherwise.  Query head h reads kv head h / (q_heads / kv_heads).
 *   out = sum softmax(scale * q.k) v     lse = ln sum exp(scale * q.k)
 * A prefix's rows are computed once for all rows of its group.  A query that
 * sees no key gets zeros and lse = -inf.  Keys whose page-table index or page
 * id is out of range are not seen, whatever memory holds, and are counted in
 * *skipped (if not NULL): once per request with query tokens for a context,
 * once per group with query tokens for a prefix.  Values outside what a query
 * sees never reach its output, infinities and NaN included.  tok_off[num_reqs]
 * may be less than total_tokens here: rows of q from there on are not read, and
 * those of out and lse keep their contents, so that one captured call serves
 * batches of up to total_tokens.  A sum over more
 * keys than one workgroup takes is joined in an order that depends on the
 * lengths alone (over a KVX_FP4 pool also on the tables' num_ids, from which the
 * kernel for small or large batches is chosen), so results repeat bit for bit.
 *
 * The pool holds the type of q, KVX_FP8 (e4m3) or KVX_FP4; f32 pools, num_kv = 1
 * and head_dim above 256 are KVX_E_UNSUPPORTED.  head_dim * element size is a
 * multiple of 16.  Values of KVX_FP4 pools take part as they are held; their
 * scale bytes are 104 to 140 or 255, which is what kvx_append writes (the results
 * of others are unspecified).  Products and sums are 32 bits; the softmax's weights are
 * rounded to q's type for their product with V (half a step: 2^-8 of a weight
 * in bf16, 2^-11 in f16).
 *
 * Range.  Weights are taken against a reference that may lag the maximum and
 * reach 2^8 (in bf16) before the division by their sum, so bf16 values larger
 * than 2^119 over the number of keys seen may make an infinity where their mean
 * is finite; those of f16, e4m3 and 4-bit pools cannot.  Scores of finite inputs
 * (scale * q.k * log2 e) have to stay inside +-2^127.  An infinity or a NaN among
 * the values makes an infinity or a NaN in the outputs that see it (a NaN also
 * from an infinity whose weight rounds to 0).
 *
 * The contracts of tok_off and grp_off are unchecked (KVX_VALIDATE=1 checks
 * them, and that lengths are not negative: KVX_E_SHAPE); with broken ones the
 * kernels stay inside the pool, the workspace, q, out and lse, and the result
 * is unspecified.  Negative lengths count as 0, and those past 2^30 as 2^30.  At
 * most 2^24 requests and groups and 2^23 - 1 query tokens (KVX_E_RANGE).
 *
 * No row of out may share a byte with one of q, nor lse or the workspace with
 * either or each other (KVX_E_OVERLAP); slices of one fused buffer are fine.
 *
 * The workspace holds partial sums during the call and nothing between calls.
 * Calls that may run at the same time, graph replays among them, need a
 * workspace each.  kvx_attend_workspace gives the bytes for a batch of at most
 * this many requests, groups and tokens.  Two launches. */
kvx_status kvx_attend(const kvx_layout* layout, int32_t layer, const kvx_pool* pool,
                      int32_t block_layout, const kvx_reqs* reqs, const int32_t* ctx_len,
                      const kvx_table* table, const kvx_prefix* prefix,
                      const kvx_attention* attention, unsigned long long* skipped,
                      hipStream_t stream);

kvx_status kvx_attend_workspace(const kvx_layout* layout, int32_t num_reqs, int32_t num_groups,
                                int64_t total_tokens, int32_t q_heads, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* KVX_SERVE_H */
