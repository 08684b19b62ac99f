// logprobs.hip -- log probabilities of given tokens, entropy and top
// alternatives of each row of logits.
#include "serving.h"

namespace cl {
namespace {

struct LogprobArgs {
  const void* x;
  int64_t x_row;
  const int32_t* ids;
  float* logp;
  float* entropy;
  int32_t* top_ids;
  float* top_logp;
  int rows, vocab, given, top_k;
};

// Order of the alternatives as one number: larger logits first (-0 as +0, NaN largest), then lower ids.
__device__ __forceinline__ uint64_t rank_key(float x, int id) {
  uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  if (x != x) u = 0x7FFFFFFFu;
  u = (u >> 31) ? ~u : u | 0x80000000u;
  return (uint64_t)u << 32 | (uint32_t)~id;
}

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, T* lds, F f) {
  for (int d = 1; d < 64; d <<= 1) v = f(v, __shfl_xor(v, d));
  __syncthreads();
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  v = lds[0];
  for (int w = 1; w < 4; ++w) v = f(v, lds[w]);
  return v;
}

// One workgroup a row: maximum, sums, then top_k rounds that each find the largest key below the last.
template <int DT>
__global__ void __launch_bounds__(256) logprobs_kernel(LogprobArgs a) {
  __shared__ float lds_f[4];
  __shared__ unsigned long long lds_u[4];
  const int t = blockIdx.x, tid = threadIdx.x;
  const auto* x = static_cast<const typename Elem<DT>::raw*>(a.x) + t * a.x_row;
  const auto add = [](float p, float q) { return p + q; };
  float m = -INFINITY;
  bool nan = false;
  for (int j = tid; j < a.vocab; j += 256) {
    const float v = Elem<DT>::up(x[j]);
    nan |= v != v;
    m = fmaxf(m, v);
  }
  m = block_reduce(m, lds_f, [](float p, float q) { return fmaxf(p, q); });
  if (block_reduce(nan ? 1.f : 0.f, lds_f, add) > 0.f) m = __builtin_nanf("");
  float l = 0.f, w = 0.f;
  for (int j = tid; j < a.vocab; j += 256) {
    const float d = Elem<DT>::up(x[j]) - m, e = expf(d);
    l += e;
    w += d == -INFINITY ? 0.f : d * e;
  }
  l = block_reduce(l, lds_f, add);
  w = block_reduce(w, lds_f, add);
  const float lse = logf(l);
  if (tid == 0) a.entropy[t] = lse - w / l;
  for (int c = tid; c < a.given; c += 256) {
    const int id = a.ids[(int64_t)t * a.given + c];
    a.logp[(int64_t)t * a.given + c] = id >= 0 && id < a.vocab ? Elem<DT>::up(x[id]) - m - lse : __builtin_nanf("");
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.top_k; ++k) {
    unsigned long long best = 0;
    for (int j = tid; j < a.vocab; j += 256) {
      const unsigned long long key = rank_key(Elem<DT>::up(x[j]), j);
      if (key < last && key > best) best = key;
    }
    best = block_reduce(best, lds_u, [](unsigned long long p, unsigned long long q) { return p > q ? p : q; });
    if (tid == 0) {
      const int id = (int)~(uint32_t)best;
      a.top_ids[(int64_t)t * a.top_k + k] = id;
      a.top_logp[(int64_t)t * a.top_k + k] = Elem<DT>::up(x[id]) - m - lse;
    }
    last = best;
  }
}

}  // namespace
}  // namespace cl

using namespace cl;

extern "C" size_t cl_token_logprobs_work_bytes(int32_t rows, int32_t vocab, int32_t top_k) {
  (void)rows, (void)vocab, (void)top_k;
  return 0;
}

extern "C" cl_status cl_token_logprobs(const void* x, int32_t dtype, int64_t x_row, int32_t rows, int32_t vocab,
                                       const int32_t* ids, int32_t given, float* logp, float* entropy, int32_t top_k,
                                       int32_t* top_ids, float* top_logp, void* work, size_t work_bytes, void* stream) {
  clear_error();
  if (rows < 0 || vocab < 1 || given < 0 || top_k < 0) return fail(CL_EINVAL, "logprobs: a size is out of range");
  if (!elem_ok(dtype)) return fail(CL_EINVAL, "logprobs: unknown element type");
  if (vocab > (1 << 24)) return fail(CL_ESIZE, "logprobs: vocab above 2^24");
  if (top_k > 32) return fail(CL_EUNSUPPORTED, "logprobs: top_k %d above 32", top_k);
  if (top_k > vocab) return fail(CL_EINVAL, "logprobs: top_k %d above vocab %d", top_k, vocab);
  if (rows == 0) return CL_OK;
  if (!x || !entropy || (given && (!ids || !logp)) || (top_k && (!top_ids || !top_logp)))
    return fail(CL_EINVAL, "logprobs: a required pointer is NULL");
  if (!aligned_to(x, elem_size(dtype))) return fail(CL_EINVAL, "logprobs: x is misaligned for its type");
  (void)work, (void)work_bytes;
  const LogprobArgs a = {x, x_row, ids, logp, entropy, top_ids, top_logp, rows, vocab, given, top_k};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == CL_F16)
    hipLaunchKernelGGL((logprobs_kernel<CL_F16>), dim3(rows), dim3(256), 0, s, a);
  else if (dtype == CL_BF16)
    hipLaunchKernelGGL((logprobs_kernel<CL_BF16>), dim3(rows), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((logprobs_kernel<CL_F32>), dim3(rows), dim3(256), 0, s, a);
  return launched("logprobs");
}
