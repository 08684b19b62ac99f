/*
 * cl_serving.h -- C ABI of the operators around the compressed linear layers of
 * a decoder on MI355X (gfx950): rotary positions, the quantised K/V cache,
 * attention of drafted tokens over that cache, and log probabilities of given
 * tokens.  Together they are the step that verifies a tree of drafted tokens;
 * one new token per sequence is its smallest form.
 *
 * Conventions are those of compressed_linear.h: status codes (the message in
 * cl_last_error), device pointers the caller owns, streams as void*, work
 * asynchronous on the stream, nothing allocated, every entry recordable into a
 * HIP graph.  The launch goes to the current HIP device.  Strides count
 * elements; the channels of a head are contiguous.  A call with no tokens
 * returns CL_OK and launches nothing.
 */
#ifndef CL_SERVING_H
#define CL_SERVING_H

#include "compressed_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { CL_F16 = 0, CL_BF16 = 1, CL_F32 = 2 } cl_dtype;
/* Pairs of a rotation over `rot` channels: HALF (i, i + rot/2), INTERLEAVED (2i, 2i + 1). */
typedef enum { CL_ROPE_HALF = 0, CL_ROPE_INTERLEAVED = 1 } cl_rope_layout;
/* Which axis a pair belongs to, where positions have several: BLOCKS the pairs of an axis lie side by side, TURNS the axes alternate. */
typedef enum { CL_ROPE_BLOCKS = 0, CL_ROPE_TURNS = 1 } cl_rope_order;
/* How rotation angles are scaled for contexts past the trained length. */
typedef enum { CL_ROPE_NONE = 0, CL_ROPE_LINEAR = 1, CL_ROPE_NTK = 2, CL_ROPE_YARN = 3 } cl_rope_scaling;
typedef enum { CL_KV_INT8 = 0, CL_KV_INT4 = 1 } cl_kv_kind;

/*
 * cl_rope_table -- cosines and sines of every position and pair.
 *   table    device, [positions, rot / 2, 2] fp32, overwritten: (cos a, sin a) * m, computed in
 *            fp64 and rounded once, with a = p * w_i and w_i = base^(-2i/rot) changed by
 *   scaling  NONE    m = 1
 *            LINEAR  w_i / factor, m = 1
 *            NTK     base replaced by base * factor^(rot / (rot - 2)), m = 1 (rot >= 4)
 *            YARN    w_i * (1 - g_i) / factor + w_i * g_i, where g_i falls linearly in i from 1 to 0
 *                    between the pairs that turn beta_fast and beta_slow times within `trained`
 *                    positions (floor of the first index, ceiling of the second, kept in [0, rot - 1],
 *                    at least 0.001 apart); m = 0.1 ln(factor) + 1
 *   factor >= 1; trained, beta_fast > beta_slow > 0 are read by YARN only.
 * Errors: CL_EINVAL (sizes, rot odd, NULL or misaligned table, parameters), CL_EHIP.
 */
cl_status cl_rope_table(int32_t positions, int32_t rot, double base, int32_t scaling, double factor, int32_t trained,
                        double beta_fast, double beta_slow, float* table, void* stream);

/*
 * cl_rope -- rotary positions: for each pair (x1, x2) of the first `rot` channels of a head and the
 * pair's (c, s) in the table row of its token's position,
 *     y1 = x1 c - x2 s        y2 = x2 c + x1 s
 * in fp32, each product and each sum rounded, then rounded once to the output type.  The channels from
 * `rot` on are copied.
 *   x, x_dtype            device, [tokens, heads, dim], strides x_token, x_head
 *   positions             device, [tokens] int32; a position outside [0, table_rows) gives NaN in
 *                         the rotated channels
 *   table, table_rows     device, [table_rows, rot / 2, 2] fp32, 8-byte aligned
 *   y, y_dtype            device, [tokens, heads, dim], strides y_token, y_head.  y may be x (same
 *                         type and strides); otherwise the two must not overlap.
 * Errors: CL_EINVAL (sizes, rot odd or not in [2, dim], unknown type or layout, NULL pointers, an address
 * that is no multiple of its element), CL_ESIZE (dim > 1024, tokens * heads * dim >= 2^40, heads * dim >= 2^33), CL_EHIP.
 */
cl_status cl_rope(const void* x, int32_t x_dtype, int64_t x_token, int64_t x_head, int32_t tokens, int32_t heads,
                  int32_t dim, const int32_t* positions, const float* table, int32_t table_rows, int32_t rot,
                  int32_t layout, void* y, int32_t y_dtype, int64_t y_token, int64_t y_head, void* stream);

/*
 * cl_rope_axes -- cl_rope for positions with several axes (time, height and width of a video, say): pair i of a
 * token is rotated by the table row of the token's position on the pair's axis a(i).
 *   positions        device, [axes, tokens] int32; a position outside [0, table_rows) gives NaN in the pairs of its
 *                    axis
 *   axes, sections   1 to 4; host, [axes] int32, the pairs of each axis (0 is allowed), rot / 2 together.
 *                    sections NULL: one axis, the others are not read
 *   order            BLOCKS  the first sections[0] pairs belong to axis 0, the next sections[1] to axis 1, and so on;
 *                    TURNS   a(i) = i % axes while i / axes < sections[i % axes], otherwise axis 0
 * A table whose frequencies start anew with each axis (an image's height and width) is one whose columns are those of
 * several cl_rope_table side by side.
 * Errors: as cl_rope; CL_EINVAL for sections that are negative, do not add up to rot / 2, or do not get all their
 * turns.
 */
cl_status cl_rope_axes(const void* x, int32_t x_dtype, int64_t x_token, int64_t x_head, int32_t tokens, int32_t heads,
                       int32_t dim, const int32_t* positions, int32_t axes, const int32_t* sections, int32_t order,
                       const float* table, int32_t table_rows, int32_t rot, int32_t layout, void* y, int32_t y_dtype,
                       int64_t y_token, int64_t y_head, void* stream);

/*
 * A paged, quantised K/V cache in caller-owned device memory.  Slot s is place s % page_size of page
 * s / page_size.
 *   INT8  k, v [pages, heads, page_size, dim] bytes, byte = code + 128, code in -127..127;
 *         k_scale, v_scale [pages, heads, page_size] fp16, one scale to a (token, head);
 *   INT4  k, v [pages, heads, page_size, dim / 2] bytes, nibble = code + 8, code in -7..7, channel 2i in
 *         the low nibble of byte i; k_scale, v_scale [pages, heads, page_size, dim / 32] fp16, one scale to
 *         32 channels.
 * A stored value is code * scale.  Scales are finite; an int4 scale has at most 8 significant bits, so
 * that code * scale is an fp16 value.  page_size is a power of two in [16, 1024]; dim is 64 or 128;
 * pages * page_size < 2^31; k and v 16-byte aligned, scales 8-byte aligned.  Memory that was never
 * written may hold anything: it is not read as a value.
 */
typedef struct {
  void* k;
  void* v;
  uint16_t* k_scale;
  uint16_t* v_scale;
  int32_t pages, page_size, heads, dim;
  int32_t kind;      /* cl_kv_kind */
  int32_t reserved;  /* 0 */
} cl_kv_cache;

/*
 * cl_kv_append -- quantise the keys and values of new tokens into the cache.
 *   k, v, dtype      device, [tokens, heads, dim], strides k_token, k_head and v_token, v_head
 *   slots            device, [tokens] int32; a slot outside [0, pages * page_size) (-1, say) stores nothing.
 *                    No two tokens of a call may have the same slot.
 *   positions, table, table_rows, rot, layout
 *                    as in cl_rope: the keys are rotated on the way, from unrounded fp32 results; table NULL:
 *                    they are taken as they are.  A key whose position lies outside the table is stored
 *                    as zeros.
 * With a = max |value| over the scale's channels (a NaN counts as 0, an infinity saturates):
 *   INT8  scale = fp16(min(a / 127, 65504)), code = clamp(rint(value * (1 / scale)), -127, 127)
 *   INT4  scale = fp16(bf16(min(a / 7, 8192))), code = clamp(rint(value * (1 / scale)), -7, 7)
 * every step rounded to nearest-even in fp32; a zero scale has codes 0.
 * Errors: CL_EINVAL (as cl_rope, a malformed cache), CL_EUNSUPPORTED (dim), CL_ESIZE, CL_EHIP.
 */
cl_status cl_kv_append(const cl_kv_cache* cache, const void* k, const void* v, int32_t dtype, int32_t tokens,
                       int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, const int32_t* slots,
                       const int32_t* positions, const float* table, int32_t table_rows, int32_t rot, int32_t layout,
                       void* stream);

/*
 * cl_kv_append_axes -- cl_kv_append for positions with several axes; positions, axes, sections, order as in
 * cl_rope_axes.  A key with a position outside the table on an axis that has pairs is stored as zeros.
 * Errors: as cl_kv_append and cl_rope_axes.
 */
cl_status cl_kv_append_axes(const cl_kv_cache* cache, const void* k, const void* v, int32_t dtype, int32_t tokens,
                            int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, const int32_t* slots,
                            const int32_t* positions, int32_t axes, const int32_t* sections, int32_t order,
                            const float* table, int32_t table_rows, int32_t rot, int32_t layout, void* stream);

/*
 * cl_kv_read -- the stored values of n slots: k_out[i], v_out[i] [heads, dim] = code * scale of slot
 * slots[i], rounded once to `dtype`; zeros for a slot outside the cache.
 *   k_out, v_out     device, [n, heads, dim] contiguous, 16-byte aligned; slots device, [n] int32.
 * Errors: as cl_kv_append.
 */
cl_status cl_kv_read(const cl_kv_cache* cache, const int32_t* slots, int32_t n, void* k_out, void* v_out,
                     int32_t dtype, void* stream);

/*
 * cl_kv_copy_pages -- whole pages copied inside a cache: page src[i] to page dst[i], codes and scales of K and V.
 *   src, dst         device, [n] int32.  An entry with either outside [0, pages) (-1, say) copies nothing.  No page is the
 *                    destination of two entries, or of one and the source of another.
 * Scales must be 16-byte aligned.
 * Errors: CL_EINVAL (a malformed cache, n < 0, NULL or misaligned pointers), CL_EUNSUPPORTED (dim), CL_ESIZE, CL_EHIP.
 */
cl_status cl_kv_copy_pages(const cl_kv_cache* cache, const int32_t* src, const int32_t* dst, int32_t n, void* stream);

/*
 * cl_kv_keep -- accepted drafts moved together.  Sequence b has ctx_lens[b] tokens, followed in the cache by its drafts;
 * for each j with i = kept[b][j] >= 0 the entries of draft i (place ctx_lens[b] + i) are copied to place
 * ctx_lens[b] + j, codes and scales as they are.  All of a sequence's drafts are read before any is written, so kept may be
 * any list, in any order.
 *   block_table      device, [sequences, table_width] int32, as in cl_tree_attention
 *   ctx_lens, kept   device, [sequences] and [sequences, most] int32, most <= 256
 * A place past the table's width or whose page lies outside the cache is neither read nor written.  The places
 * written belong to their sequence alone (cl_pool_extend sees to that).
 * Errors: CL_EINVAL, CL_EUNSUPPORTED (dim, most), CL_ESIZE, CL_EHIP.
 */
cl_status cl_kv_keep(const cl_kv_cache* cache, const int32_t* block_table, int32_t table_width, int32_t sequences,
                     const int32_t* ctx_lens, const int32_t* kept, int32_t most, void* stream);

/*
 * Which sequence holds which pages, in caller-owned device memory.  The pages are numbers: any caches of the same page
 * size (a model's layers, say) share a pool.
 *   block_table      [sequences, width] int32: a sequence's pages in their order, -1 past the last
 *   lens             [sequences] int32: its tokens
 *   refs             [pages] int32: how many times a page stands in the table; 0: it is free
 *   left_out         [1] int32, written by cl_pool_extend
 * A sequence of n tokens has ceil(n / page_size) pages.  At the start the table is -1, lens and refs 0.  A program
 * may hold a page itself by adding to its refs.
 * page_size is a power of two in [16, 1024]; sequences <= 4096; pages * page_size and width * page_size < 2^31.  One
 * call at a time may use a pool; its operations and everything that reads it run in the stream's order.
 */
typedef struct {
  int32_t* block_table;
  int32_t* lens;
  int32_t* refs;
  int32_t* left_out;
  int32_t sequences, width, pages, page_size;
} cl_page_pool;

/*
 * cl_pool_extend -- room for new tokens: sequence b gets n_b = cu_q[b+1] - cu_q[b] more, and pages for them, its last page
 * among them if other sequences hold that too and its tokens do not fill it (it has to be copied then).  Of a
 * page whose holders are all extended the last one keeps it.  Free pages are given out lowest first, to
 * sequences in their order and to each one's places in their order.
 *   cu_q             device, [sequences + 1] int32, as in cl_tree_attention
 *   slots            device, [tokens] int32: the new tokens' slots, for cl_kv_append; -1 for tokens of no sequence and
 *                    of those left out
 *   src, dst         device, [sequences] int32: the page to copy (cl_kv_copy_pages, in every cache, before anything is
 *                    appended), -1 where there is none
 * A sequence whose cu_q does not fit [0, tokens] or begins below an earlier number of cu_q, whose table is too narrow or whose
 * last page is no page is left out and stays as it was; so is one for which the free pages do not suffice, and every one after it that gets tokens.
 * left_out is how many there are.
 * Errors: CL_EINVAL, CL_ESIZE, CL_EHIP.
 */
cl_status cl_pool_extend(const cl_page_pool* pool, const int32_t* cu_q, int32_t tokens, int32_t* slots, int32_t* src,
                         int32_t* dst, void* stream);

/*
 * cl_pool_fork -- every sequence b at once becomes what sequence parents[b] was, sharing its pages: parents[b] == b
 * stays, -1 (any number that is no sequence) ends and gives its pages back.
 *   parents          device, [sequences] int32
 * Errors: CL_EINVAL, CL_ESIZE, CL_EHIP.
 */
cl_status cl_pool_fork(const cl_page_pool* pool, const int32_t* parents, void* stream);

/*
 * cl_pool_truncate -- sequences shortened to lens[b] tokens, the pages past them given back; a negative number or
 * one that is not below the sequence's leaves it.
 *   lens             device, [sequences] int32, not the pool's own
 * Errors: CL_EINVAL, CL_ESIZE, CL_EHIP.
 */
cl_status cl_pool_truncate(const cl_page_pool* pool, const int32_t* lens, void* stream);

/*
 * cl_pool_compact -- the highest pages that are held move to the lowest free ones, while those are lower: after enough moves
 * the n pages that are held are 0 to n - 1.  The table and refs are changed; the pages are to be copied
 * (cl_kv_copy_pages, in every cache).
 *   max_moves        at most this many pages move
 *   src, dst         device, [max_moves] int32: the moves, highest source first; -1 past the last
 *   work             device, cl_pool_compact_work_bytes(pages) bytes
 * Errors: CL_EINVAL, CL_ESIZE, CL_ENOMEM (work_bytes too small), CL_EHIP.
 */
size_t cl_pool_compact_work_bytes(int32_t pages);
cl_status cl_pool_compact(const cl_page_pool* pool, int32_t max_moves, int32_t* src, int32_t* dst, void* work,
                          size_t work_bytes, void* stream);

/*
 * cl_tree_attention -- attention of each sequence's newest tokens over its cached keys and values.
 * Sequence b has ctx_lens[b] cached tokens, followed in the cache by its n_b = cu_q[b+1] - cu_q[b] new
 * tokens (already appended): cached token j lies in place j % page_size of page
 * block_table[b][j / page_size].  New token t sees the ctx_lens[b] tokens before and, of the new
 * ones, those whose bit is set in its mask:
 *     o = sum_j p_j v_j,   p = softmax_j(scale * q . k_j)      over the tokens it sees
 * and zeros where it sees none.  Query head h reads kv head h / (q_heads / heads).
 *   q, o, dtype      device, [cu_q[sequences], q_heads, dim] fp16 or bf16 (16-byte aligned, strides
 *                    multiples of 8 elements); q strides q_token, q_head; o contiguous, same type.
 *   tokens           rows of q and o (cu_q[sequences])
 *   block_table      device, [sequences, table_width] int32
 *   ctx_lens, cu_q   device, [sequences] and [sequences + 1] int32; cu_q starts at 0, nondecreasing
 *   max_q            at least every n_b, at most 256
 *   max_ctx          the longest ctx_lens; sizes the launch.  Longer ones are still computed rightly.
 *   mask             device, [tokens, mask_words] int64, bit i of a row's words: new token i is seen.
 *                    NULL: token t sees new tokens 0..t.  mask_words >= ceil(max_q / 64); bits from n_b on
 *                    are ignored.
 *   scale            of the scores, finite
 *   work             device, cl_tree_attention_work_bytes(...) bytes for these arguments, 16-byte aligned (may be
 *                    NULL where that is 0; never more than CL_ATTENTION_COUNTER_BYTES + 2^29).  Its first
 *                    CL_ATTENTION_COUNTER_BYTES are zeroed once before its first use; calls leave them zeroed.  One
 *                    call at a time may use it.
 * Scores, maxima, sums and outputs are held in fp32; keys and values enter the matrix cores exactly, and queries as fp16,
 * each row scaled by a power of two: channels below 2^-27 of the row's largest are kept to 2^-38 of it.  The
 * probabilities (int8: times V's scale) enter them as fp16, scaled so that those down to 2^-24 of the largest
 * (int8: of the largest probability times the largest V scale that the row has seen so far) keep fp16's
 * 11 bits; below 2^-35 of it they are lost.
 * A page of block_table outside the cache, or a place past its width, gives NaN in the rows that see it.
 * Tokens that a row does not see do not change its bits, whatever their codes and scales are in memory, if no row
 * of the call sees them or their scales are finite: a drafted token may have been stored nowhere (slot -1).
 * Sequences whose cu_q does not fit [0, tokens] or max_q are left out: their rows, and those from cu_q[sequences] on, are
 * not written.
 * Deterministic: the same inputs give bitwise identical o.
 * Errors: CL_EINVAL, CL_EUNSUPPORTED (dim, max_q > 256), CL_ESIZE, CL_ENOMEM (work_bytes too small), CL_EHIP.
 */
#define CL_ATTENTION_COUNTER_BYTES 262144
size_t cl_tree_attention_work_bytes(int32_t sequences, int32_t q_heads, int32_t heads, int32_t dim, int32_t max_q,
                                    int32_t max_ctx);
cl_status cl_tree_attention(const void* q, int32_t dtype, int64_t q_token, int64_t q_head, int32_t tokens,
                            int32_t q_heads, const cl_kv_cache* cache, const int32_t* block_table, int32_t table_width,
                            int32_t sequences, const int32_t* ctx_lens, const int32_t* cu_q, int32_t max_q,
                            int32_t max_ctx, const int64_t* mask, int32_t mask_words, float scale, void* o, void* work,
                            size_t work_bytes, void* stream);

/*
 * cl_recording -- the number of the graph recording that `stream` is part of (HIP gives each its own), 0
 * if it is not recorded.  For callers that keep a workspace to a recording: what clears it runs with the
 * replays, which may run on any stream next to other calls.
 * Errors: CL_EINVAL (id NULL), CL_EHIP.
 */
cl_status cl_recording(void* stream, uint64_t* id);

/*
 * cl_token_logprobs -- log probabilities of given tokens, entropy and top alternatives of each row of
 * logits.  With m = max_j x_j and l = sum_j exp(x_j - m):
 *     logp[t, c] = x[ids[t, c]] - m - log l                     NaN for an id outside [0, vocab)
 *     entropy[t] = log l - sum_j (x_j - m) exp(x_j - m) / l     a logit of -inf adds nothing
 *     top_ids[t], top_logp[t]: the top_k logits, largest first, equal ones by the lower id (-0 equals +0, a NaN
 *     is the largest)
 * in fp32.  A row with a NaN or +inf gives NaN where the formula does; a row of -inf only has logp NaN.
 *   x, dtype         device, [rows, vocab], row stride x_row
 *   ids              device, [rows, given] int32 (given may be 0)
 *   logp, entropy    device, [rows, given] and [rows] fp32
 *   top_ids, top_logp  device, [rows, top_k] int32 and fp32 (NULL if top_k is 0); 0 <= top_k <= min(32, vocab)
 * Errors: CL_EINVAL, CL_EUNSUPPORTED (top_k > 32), CL_ESIZE (vocab > 2^24), CL_EHIP.
 */
cl_status cl_token_logprobs(const void* x, int32_t dtype, int64_t x_row, int32_t rows, int32_t vocab,
                            const int32_t* ids, int32_t given, float* logp, float* entropy, int32_t top_k,
                            int32_t* top_ids, float* top_logp, void* stream);

/*
 * cl_call -- calls cl_rope, cl_kv_append, cl_kv_read, cl_tree_attention, cl_token_logprobs or an entry of the second list with
 * its arguments in an array, in their order: pointers and integers as 64-bit integers, a float as the bits of a
 * double.  For bindings that pay for every argument of a foreign call.
 * Errors: the entry's; CL_EINVAL for an unknown entry or args NULL.
 */
enum { CL_CALL_ROPE = 0, CL_CALL_KV_APPEND = 1, CL_CALL_KV_READ = 2, CL_CALL_TREE_ATTENTION = 3, CL_CALL_TOKEN_LOGPROBS = 4 };
enum { CL_CALL_ROPE_AXES = 16, CL_CALL_KV_APPEND_AXES = 17, CL_CALL_KV_COPY_PAGES = 18, CL_CALL_KV_KEEP = 19,
       CL_CALL_POOL_EXTEND = 20, CL_CALL_POOL_FORK = 21, CL_CALL_POOL_TRUNCATE = 22, CL_CALL_POOL_COMPACT = 23,
       CL_CALL_INT8_QUANT = 24, CL_CALL_INT8_LINEAR = 25, CL_CALL_INT8_FORWARD = 26 /* cl_int8.h */ };
cl_status cl_call(int32_t entry, const int64_t* args);

#ifdef __cplusplus
}
#endif
#endif
