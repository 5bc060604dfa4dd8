/*
 * ctcpb_lm.h -- C ABI of libctcpb_lm.so: the operators a language model needs
 * to rescore the decoder's N-best lists on AMD Instinct MI355X (gfx950).
 *
 *   cache_plan / cache_release   page tables and slot maps of a paged
 *                                key/value cache, from device-resident lengths
 *   cache_store                  new tokens' keys and values to their slots
 *   attention                    one new token per request over the cache
 *   loss / loss_grad             token losses over a large vocabulary without
 *                                keeping the logits, and their gradients
 *
 * Conventions are those of ctcpb.h: device pointers are the caller's, the
 * library allocates no device memory and keeps no state between calls, every
 * call only enqueues work on `stream` (a hipStream_t, NULL = the default
 * stream) and may be captured into a HIP graph.  The return value is CTCPB_OK
 * or an error code (the values of ctcpb.h), described by
 * ctcpb_lm_last_error().  On error nothing was enqueued, except
 * CTCPB_ERR_DEVICE, reported when a launch fails.  Each call takes its operands
 * in a structure that it reads before it returns.  Strides are in elements.
 * Elements of a tensor that is written must not share memory.
 * Results do not depend on the order in which workgroups run: two calls on the
 * same inputs give the same bits.
 */
#ifndef CTCPB_LM_H
#define CTCPB_LM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the tensors documented "typed". */
enum { CTCPB_LM_BF16 = 0, CTCPB_LM_F16 = 1, CTCPB_LM_F32 = 2 };

/* Added to the dtype of ctcpb_lm_loss_grad and its size query: d as the sum of two
 * values of a 16-bit type, see there.  Of no account with CTCPB_LM_F32. */
enum { CTCPB_LM_SPLIT_D = 256 };

/* Status bits of ctcpb_lm_cache_plan. */
enum {
  CTCPB_LM_NO_PAGE = 1,   /* the pool ran out before the row had its pages */
  CTCPB_LM_NO_ENTRY = 2,  /* the row's table is full */
  CTCPB_LM_NO_SLOT = 4    /* the slot map is full: the row's last tokens were left out */
};

/* Hand out pages for counts[r] new tokens of every request r that already
 * holds lengths[r] tokens, and list the slots of the new tokens.
 *   lengths, counts  device int32 [rows]; negative values count as 0, lengths
 *                    are clamped to table_width * page_size
 *   tables           device int32 [rows][table_width] with row stride
 *                    table_stride: entry p of row r is the page of the row's
 *                    tokens p*page_size ..; entries of pages the row holds are
 *                    read, the entries of new pages are written (-1 where the
 *                    pool has none left), the others are left alone
 *   pool, taken      device int32 [pool_size] free page ids (distinct, >= 0)
 *                    and int32 [1], how many of them are in use: pages are
 *                    taken from pool[taken] on, in row order, then page order
 *   page_size        a power of two in 4..256
 *   slots, positions device int32 [capacity]: for the new tokens, rows in
 *                    order, the slot (page * page_size + offset; -1 if the
 *                    token has no page) and the position in its request;
 *                    entries past the last token are -1
 *   starts           device int32 [rows + 1]: row r's new tokens are
 *                    slots[starts[r]] ..; a sum above 2^30 counts as 2^30.
 *                    A row's tokens past `capacity` are not appended.
 *   out_lengths      device int32 [rows]: tokens with a slot, old and new
 *   out_taken        device int32 [1]
 *   status           device int32 [rows]: CTCPB_LM_NO_* bits, 0 = complete
 * slots, positions, starts, out_lengths, out_taken and status must not overlap
 * the inputs, so a repeated call on the same inputs gives the same result.
 * num_pages * page_size, with num_pages the largest page id + 1, must be below
 * 2^31. */
typedef struct {
  const int32_t *lengths, *counts;
  int32_t* tables;
  const int32_t *pool, *taken;
  int32_t *slots, *positions, *starts, *out_lengths, *out_taken, *status;
  int64_t table_stride;
  int32_t rows, table_width, pool_size, page_size, capacity;
} ctcpb_lm_plan_args;
int ctcpb_lm_cache_plan(const ctcpb_lm_plan_args* args, void* stream);

/* Give back the pages of the rows with finished[r] != 0 (device uint8 [rows]):
 * they go to pool[out_taken ..] in row order, then page order, and
 * out_taken = taken - (their number).  out_lengths is 0 for these rows,
 * lengths[r] for the others.  Other arguments as ctcpb_lm_cache_plan; out_*
 * must not overlap the inputs. */
typedef struct {
  const uint8_t* finished;
  const int32_t *lengths, *tables;
  int32_t* pool;
  const int32_t* taken;
  int32_t *out_lengths, *out_taken;
  int64_t table_stride;
  int32_t rows, table_width, pool_size, page_size;
} ctcpb_lm_release_args;
int ctcpb_lm_cache_release(const ctcpb_lm_release_args* args, void* stream);

/* A paged cache tensor: element (page, offset, head, d) at
 * data[page*stride_page + offset*stride_token + head*stride_head + d].  The
 * order of the axes in memory is free (token by token or head by head). */
typedef struct {
  void* data;            /* device, typed */
  int64_t stride_page, stride_token, stride_head;
} ctcpb_lm_cache;

/* Write the keys and values of `tokens` tokens to their slots.
 *   k, v     device, typed: element (t, head, d) at t*stride_t + head*stride_h + d
 *   slots    device int32 [tokens]; tokens whose slot is outside
 *            [0, num_pages*page_size) are left out.  Slots are distinct.
 * 16-byte accesses are used where pointers and strides allow, else single
 * elements. */
typedef struct {
  const void *k, *v;
  const int32_t* slots;
  int64_t k_stride_t, k_stride_h, v_stride_t, v_stride_h;
  ctcpb_lm_cache k_cache, v_cache;
  int32_t dtype, tokens, num_pages, page_size, kv_heads, head_dim;
} ctcpb_lm_store_args;
int ctcpb_lm_cache_store(const ctcpb_lm_store_args* args, void* stream);

/* Attention of one token per request over its pages (the token's own key and
 * value stored before).  With t over the last `window` of the request's
 * lengths[r] tokens (window 0: all of them), kv = head / (q_heads / kv_heads):
 *   s_t = scale * q[r, head] . k[t, kv]      m = max s_t     l = sum exp(s_t - m)
 *   out[r, head] = sum exp(s_t - m) v[t, kv] / l        lse[r, head] = m + log l
 * A row with no token, or with every s_t = -inf, gives zeros and lse = -inf.
 * Slots past a row's length are never used, whatever they hold.  Values within it
 * have to be finite with 16-bit types (probabilities are two numbers there, one of
 * which may be 0: an infinite value gives NaN).
 *   q, out   device, typed, element (r, head, d) at r*stride_r + head*stride_h + d
 *   lse      device float32 [rows][q_heads], or NULL
 *   tables   as ctcpb_lm_cache_plan leaves them; entries are clamped to the cache
 *   lengths  device int32 [rows], clamped to [0, min(max_len, table_width*page_size)]
 *   max_len  an upper bound of the lengths that the caller knows (it sizes the
 *            launch), 0: table_width * page_size
 *   head_dim a multiple of 8, at most 256; caches 16-byte aligned, with strides
 *            that are multiples of 16 bytes
 *   workspace  device, >= ctcpb_lm_attention_workspace bytes, 16-byte aligned;
 *            its contents on entry do not matter; calls that share it must not
 *            overlap.  */
typedef struct {
  const void* q;
  const int32_t *tables, *lengths;
  void* out;
  float* lse;
  int64_t q_stride_r, q_stride_h, out_stride_r, out_stride_h, table_stride;
  ctcpb_lm_cache k_cache, v_cache;
  int32_t dtype, rows, q_heads, kv_heads, head_dim, num_pages, page_size, table_width, max_len,
      window;
  float scale;
} ctcpb_lm_attention_args;
/* Reads no pointer of `args`, only sizes. */
int ctcpb_lm_attention_workspace(const ctcpb_lm_attention_args* args, size_t* out_bytes);
int ctcpb_lm_attention(const ctcpb_lm_attention_args* args, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Token losses of an output layer, the vocabulary taken in pieces:
 *   logit[n, v] = x[n] . w[v] + bias[v]     lse[n] = log sum_v exp(logit[n, v])
 *   loss[n] = lse[n] - logit[n, targets[n]]
 * A target outside [0, vocab) (the decoder's -1 padding) gives loss 0.
 *   x, w     device, typed, row strides stride_x / stride_w >= hidden, unit
 *            stride over `hidden`
 *   bias     device float32 [vocab], or NULL
 *   targets  device int32 [rows];  loss, lse: device float32 [rows]
 * Products of 16-bit types are summed in float32; float32 inputs are
 * multiplied in float32.  workspace: device, 256-byte aligned, contents on
 * entry do not matter; calls that share it must not overlap.  Its size depends
 * on the addresses and strides of x and w (rows that are not 16-byte aligned
 * are copied to aligned ones there); the size query does not read them. */
typedef struct {
  const void *x, *w;
  const float* bias;
  const int32_t* targets;
  float *loss, *lse;
  int64_t stride_x, stride_w;
  int32_t dtype, rows, vocab, hidden;
} ctcpb_lm_loss_args;
int ctcpb_lm_loss_workspace(const ctcpb_lm_loss_args* args, size_t* out_bytes);
int ctcpb_lm_loss(const ctcpb_lm_loss_args* args, void* workspace, size_t workspace_bytes,
                  void* stream);

/* Gradients of sum_n grad[n] * loss[n], recomputing the probabilities piece by
 * piece from lse:
 *   d[n, v] = grad[n] * (exp(logit[n, v] - lse[n]) - (v == targets[n]))
 *   dx = d w     dw = d^T x     dbias[v] = sum_n d[n, v]
 * Rows without a target have d = 0 and no part in dx and dbias, whatever their x
 * holds; for dw their x has to be finite, as 0 times infinity is NaN.
 *   grad     device float32 [rows];  lse: as ctcpb_lm_loss left it
 *   dx       device, typed [rows][hidden], contiguous;  dw: device, typed
 *            [vocab][hidden], contiguous;  dbias: device float32 [vocab].  Any
 *            of them may be NULL and is then not computed.
 * With 16-bit types d is rounded to that type before the products, scaled so
 * that the largest |grad| is a power of two (which keeps f16 in range and the
 * rounding small): the errors of dx and dw are mostly 1.0 to 1.4 times those of
 * rounding the exact results, and up to 2.2 times where most rows share a weight that
 * is not the largest (their targets' entries are then rounded alike).  For up to 64
 * rows or rows * vocab * hidden of 2^26, and at any size with CTCPB_LM_SPLIT_D, d is the
 * sum of two values of the type, and the errors are those of rounding the results; dx and dw then take twice
 * the products and d twice the room.  Sums
 * are float32.  The workspace holds up to 1 GiB of d at a time (256 columns of it
 * at least), the sums of dx if d is made in several pieces, those of products that
 * are cut along k, and those of dbias if it is not NULL: 811 MiB at 8192 x 50000 x 2048
 * bf16 without dbias, 784 of them d.  Its size depends on x and w as above, and on
 * whether dbias is NULL. */
typedef struct {
  const void *x, *w;
  const float* bias;
  const int32_t* targets;
  const float *grad, *lse;
  void *dx, *dw;
  float* dbias;
  int64_t stride_x, stride_w;
  int32_t dtype, rows, vocab, hidden;
} ctcpb_lm_grad_args;
int ctcpb_lm_loss_grad_workspace(const ctcpb_lm_grad_args* args, size_t* out_bytes);
int ctcpb_lm_loss_grad(const ctcpb_lm_grad_args* args, void* workspace, size_t workspace_bytes,
                       void* stream);

/* Human-readable description of the last error on this thread ("" if none). */
const char* ctcpb_lm_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* CTCPB_LM_H */
