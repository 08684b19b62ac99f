// tree_attention.hip -- attention of each sequence's newest tokens (a tree of
// drafted tokens; one token, a chain) over its quantised, paged K/V cache.
#include "serving.h"

namespace cl {
namespace {

struct AttnArgs {
  const uint16_t* q;
  uint16_t* o;
  cl_kv_cache c;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  const int32_t* cu_q;
  const uint64_t* mask;
  int64_t q_token, q_head;
  int tokens, q_heads, table_width, sequences, max_q, mask_words;
  float scale;
};

// One wavefront a (new token, query head); lane l holds channels 2l and 2l + 1 (dim 64: lanes 0..31).
// One pass over the keys with the running maximum and sum.
template <int DT, int KIND>
__global__ void __launch_bounds__(64) tree_attention_kernel(AttnArgs a) {
  const int b = blockIdx.z, h = blockIdx.y, t = blockIdx.x, l = threadIdx.x;
  const int first = a.cu_q[b], n_new = a.cu_q[b + 1] - first;
  if (first < 0 || n_new < 0 || n_new > a.max_q || first + n_new > a.tokens || t >= n_new) return;
  const int D = a.c.dim, hk = h / (a.q_heads / a.c.heads);
  const bool on = 2 * l < D;
  const uint16_t* q = a.q + (int64_t)(first + t) * a.q_token + (int64_t)h * a.q_head;
  const float q0 = on ? Elem<DT>::up(q[2 * l]) : 0.f, q1 = on ? Elem<DT>::up(q[2 * l + 1]) : 0.f;
  const int ctx = max(a.ctx_lens[b], 0);
  const int64_t n = (int64_t)ctx + n_new;
  float m = -INFINITY, sum = 0.f, o0 = 0.f, o1 = 0.f;
  for (int64_t j = 0; j < n; ++j) {
    if (j >= ctx) {
      const int i = (int)(j - ctx);
      const bool see = a.mask ? (a.mask[(int64_t)(first + t) * a.mask_words + i / 64] >> (i % 64)) & 1 : i <= t;
      if (!see) continue;
    }
    const int64_t pi = j / a.c.page_size;
    const int page = pi < a.table_width ? a.block_table[(int64_t)b * a.table_width + pi] : -1;
    if (page < 0 || page >= a.c.pages) {
      m = sum = o0 = o1 = __builtin_nanf("");
      break;
    }
    const int64_t row = ((int64_t)page * a.c.heads + hk) * a.c.page_size + j % a.c.page_size;
    float k0 = 0.f, k1 = 0.f, v0 = 0.f, v1 = 0.f;
    if (on) {
      const uint8_t* kb = static_cast<const uint8_t*>(a.c.k);
      const uint8_t* vb = static_cast<const uint8_t*>(a.c.v);
      if (KIND == CL_KV_INT8) {
        const float ks = Elem<CL_F16>::up(a.c.k_scale[row]), vs = Elem<CL_F16>::up(a.c.v_scale[row]);
        k0 = (float)(kb[row * D + 2 * l] - 128) * ks, k1 = (float)(kb[row * D + 2 * l + 1] - 128) * ks;
        v0 = (float)(vb[row * D + 2 * l] - 128) * vs, v1 = (float)(vb[row * D + 2 * l + 1] - 128) * vs;
      } else {
        const int64_t g = row * (D / 32) + l / 16;
        const float ks = Elem<CL_F16>::up(a.c.k_scale[g]), vs = Elem<CL_F16>::up(a.c.v_scale[g]);
        const int kk = kb[row * (D / 2) + l], vv = vb[row * (D / 2) + l];
        k0 = (float)((kk & 15) - 8) * ks, k1 = (float)((kk >> 4) - 8) * ks;
        v0 = (float)((vv & 15) - 8) * vs, v1 = (float)((vv >> 4) - 8) * vs;
      }
    }
    float s = q0 * k0 + q1 * k1;
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    s *= a.scale;
    const float up = fmaxf(m, s), old = __expf(m - up), p = __expf(s - up);
    sum = sum * old + p;
    o0 = o0 * old + p * v0;
    o1 = o1 * old + p * v1;
    m = up;
  }
  if (!on) return;
  const float r = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* o = a.o + ((int64_t)(first + t) * a.q_heads + h) * D + 2 * l;
  o[0] = Elem<DT>::down(o0 * r);
  o[1] = Elem<DT>::down(o1 * r);
}

}  // namespace
}  // namespace cl

using namespace cl;

extern "C" size_t cl_tree_attention_work_bytes(int32_t sequences, int32_t q_heads, int32_t heads, int32_t dim,
                                               int32_t max_q, int32_t max_ctx) {
  (void)sequences, (void)q_heads, (void)heads, (void)dim, (void)max_q, (void)max_ctx;
  return 0;
}

extern "C" cl_status cl_tree_attention(const void* q, int32_t dtype, int64_t q_token, int64_t q_head, int32_t tokens,
                                       int32_t q_heads, const cl_kv_cache* cache, const int32_t* block_table,
                                       int32_t table_width, int32_t sequences, const int32_t* ctx_lens,
                                       const int32_t* cu_q, int32_t max_q, int32_t max_ctx, const int64_t* mask,
                                       int32_t mask_words, float scale, void* o, void* work, size_t work_bytes,
                                       void* stream) {
  clear_error();
  cl_status st = check_cache(cache);
  if (st != CL_OK) return st;
  if (dtype != CL_F16 && dtype != CL_BF16) return fail(CL_EINVAL, "attention: q must be fp16 or bf16");
  if (tokens < 0 || sequences < 0 || max_q < 0 || max_ctx < 0) return fail(CL_EINVAL, "attention: a size is negative");
  if (q_heads < 1 || q_heads % cache->heads)
    return fail(CL_EINVAL, "attention: %d query heads over %d kv heads", q_heads, cache->heads);
  if (max_q > 256) return fail(CL_EUNSUPPORTED, "attention: max_q %d above 256", max_q);
  if (sequences > 65535 || q_heads > 65535) return fail(CL_ESIZE, "attention: more than 65535 sequences or heads");
  if (!(scale - scale == 0.f)) return fail(CL_EINVAL, "attention: scale is not finite");
  if (tokens == 0 || sequences == 0 || max_q == 0) return CL_OK;
  if (!q || !o || !block_table || !ctx_lens || !cu_q) return fail(CL_EINVAL, "attention: a required pointer is NULL");
  if (!aligned_to(q, 16) || !aligned_to(o, 16) || q_token % 8 || q_head % 8)
    return fail(CL_EINVAL, "attention: q and o must be 16-byte aligned, q's strides multiples of 8 elements");
  if (table_width < 1) return fail(CL_EINVAL, "attention: the block table has no pages");
  if (mask && mask_words < (max_q + 63) / 64)
    return fail(CL_EINVAL, "attention: %d mask words for %d new tokens", mask_words, max_q);
  (void)work, (void)work_bytes;
  const AttnArgs a = {static_cast<const uint16_t*>(q), static_cast<uint16_t*>(o), *cache, block_table, ctx_lens, cu_q,
                      reinterpret_cast<const uint64_t*>(mask), q_token, q_head, tokens, q_heads, table_width, sequences,
                      max_q, mask_words, scale};
  const dim3 grid(max_q, q_heads, sequences);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == CL_F16) {
    if (cache->kind == CL_KV_INT8)
      hipLaunchKernelGGL((tree_attention_kernel<CL_F16, CL_KV_INT8>), grid, dim3(64), 0, s, a);
    else
      hipLaunchKernelGGL((tree_attention_kernel<CL_F16, CL_KV_INT4>), grid, dim3(64), 0, s, a);
  } else {
    if (cache->kind == CL_KV_INT8)
      hipLaunchKernelGGL((tree_attention_kernel<CL_BF16, CL_KV_INT8>), grid, dim3(64), 0, s, a);
    else
      hipLaunchKernelGGL((tree_attention_kernel<CL_BF16, CL_KV_INT4>), grid, dim3(64), 0, s, a);
  }
  return launched("attention");
}
