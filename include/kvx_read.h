/*
 * kvx_read.h -- rows of a paged pool read back as dense tensors, in libkvx.so
 * beside the calls of kvx_serve.h: the inverse of kvx_append.  The conventions
 * of kvx.h and kvx_serve.h hold.
 */
#ifndef KVX_READ_H
#define KVX_READ_H

#include "kvx_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of one layer, as dense tensors.  k and v are DEVICE
 * [num_tokens][kv_heads][head_dim] tensors of `dtype`, dense in their last two
 * dimensions, their tokens k_stride and v_stride bytes apart (multiples of 16).
 * Row t of each is the row of slot slots[t] in the layer's K and V planes (NHD
 * or HND blocks); a slot may be read more than once.  Where dtype is the
 * pool's, rows are copied bit by bit and the scales are 1 (KVX_E_UNSUPPORTED
 * otherwise).  KVX_FP8 and KVX_FP4 pools are also read as f16, bf16 or f32: the
 * 32-bit products of the values with k_scale and v_scale, rounded to nearest even
 * (NaN stays NaN, what passes the type's range is an infinity).  Every scale byte
 * of a KVX_FP4 pool is read, whoever wrote it: a value is first rounded to 32 bits,
 * which the largest few pass (infinities).  Other pairs are KVX_E_UNSUPPORTED, and
 * so is KVX_FP4 as dtype.  Scales are finite, positive
 * and from 2^-64 to 2^64 (KVX_E_RANGE).  A slot outside the pool leaves its rows
 * of k and v as they were and is counted once in *skipped (if not NULL).  Rows of
 * k and v share no byte with one another (KVX_E_OVERLAP, by address), none lies in
 * a slot that the call reads (unchecked; KVX_VALIDATE=1 returns KVX_E_OVERLAP), and
 * none over the slots or the counter (unchecked).  The layout has num_kv = 2.  One launch. */
typedef struct kvx_rows_out {
    void* k;
    void* v;
    int64_t k_stride;
    int64_t v_stride;
    int64_t num_tokens;
    int32_t dtype;
    float k_scale;
    float v_scale;
} kvx_rows_out;

kvx_status kvx_read(const kvx_layout* layout, int32_t layer, const kvx_pool* pool,
                    int32_t block_layout, const int64_t* slots, const kvx_rows_out* rows,
                    unsigned long long* skipped, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVX_READ_H */
