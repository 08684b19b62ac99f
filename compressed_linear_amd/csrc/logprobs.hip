// logprobs.hip -- log probabilities of given tokens, entropy and top
// alternatives of each row of logits.
//
// One pass over a row: a thread takes 32 logits at a time into registers and
// keeps the running maximum m, l = sum exp(x - m) and w = sum (x - m) exp(x - m)
// of what it has seen (moving m by d turns w into (w - d l) e^-d, l into
// l e^-d); threads, wavefronts and, for few rows, workgroups with parts of the row
// are joined by the same rule.  log p(i) = x_i - m - log l; entropy = log l - w / l.
//
// Alternatives: a wavefront keeps its best top_k logits as 64-bit keys (order of the
// value, then of the lower id), sorted across its lanes.  One float compare of a
// logit against the last of them settles nearly every logit; the few that pass are
// inserted one by one.  A tile first raises that bar to the top_k-th largest of its
// lanes' maxima, which bounds the insertions whatever the order of the row.
//
// Bound by the read of the logits where there are rows for the whole card; a single
// row by one CU's share of it and the latency of the joins.
#include "serving.h"

namespace cl {
namespace {

constexpr int kPer = 32;  // logits of a thread's tile
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;

typedef unsigned long long u64;

struct LogprobArgs {
  const void* x;
  int64_t x_row;
  const int32_t* ids;
  float* logp;
  float* entropy;
  int32_t* top_ids;
  float* top_logp;
  int vocab, given, top_k;
};

// Order of the alternatives as one number: larger logits first (-0 as +0, NaN largest), then lower ids.
// 0 is below every key.
__device__ __forceinline__ u64 rank_key(float x, int id) {
  uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  if (x != x) u = 0x7FFFFFFFu;
  u = (u >> 31) ? ~u : u | 0x80000000u;
  return (u64)u << 32 | (uint32_t)~id;
}
__device__ __forceinline__ float key_value(u64 key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __builtin_bit_cast(float, (u >> 31) ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ u64 lane_u64(u64 v, int lane) {
  return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// Running maximum and sums of some logits.
struct Stat {
  float m, l, w;
};
__device__ __forceinline__ void join(Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  // a side without a logit above -inf has l = w = 0 and adds nothing
  const float da = a.m == m ? 0.f : a.m - m, db = b.m == m ? 0.f : b.m - m;
  const float ea = __builtin_amdgcn_exp2f(da * kLog2e), eb = __builtin_amdgcn_exp2f(db * kLog2e);
  a.w = ea * (a.w + (da == -INFINITY ? 0.f : da * a.l)) + eb * (b.w + (db == -INFINITY ? 0.f : db * b.l));
  a.l = ea * a.l + eb * b.l;
  a.m = m;
}
__device__ __forceinline__ void join_lanes(Stat& a) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) join(a, Stat{__shfl_xor(a.m, d), __shfl_xor(a.l, d), __shfl_xor(a.w, d)});
}

// A wavefront's best keys, one to a lane, largest in lane 0; lanes from `k` on are not used.
struct Best {
  u64 key;    // this lane's
  u64 last;   // the k-th: what a candidate has to beat
  float bar;  // its value; -inf until k logits have been seen
  int k;
  __device__ __forceinline__ void clear(int top_k) {
    key = last = 0;
    bar = -INFINITY;
    k = top_k;
  }
  // Inserts the keys of the lanes in `who` that beat the last one.
  __device__ __forceinline__ void insert(u64 cand, u64 who) {
    const int lane = threadIdx.x % 64;
    who &= __ballot(cand > last);
    while (who) {
      const int from = __builtin_ctzll(who);
      const u64 c = lane_u64(cand, from);
      const int at = __builtin_popcountll(__ballot(key > c));
      const int hi = __builtin_amdgcn_update_dpp(0, (int)(key >> 32), 0x138, 0xF, 0xF, false);  // from the lane below
      const int lo = __builtin_amdgcn_update_dpp(0, (int)key, 0x138, 0xF, 0xF, false);
      if (lane >= at) key = lane == at ? c : (u64)(uint32_t)hi << 32 | (uint32_t)lo;
      last = lane_u64(key, k - 1);
      who &= who - 1;
      who &= __ballot(cand > last);
    }
    bar = last ? key_value(last) : -INFINITY;
    if (bar != bar) bar = INFINITY;  // a NaN is the last: only another NaN may pass
  }
};

// A row's logits [0, j1), by a workgroup of kThreads.
template <int DT, bool VEC, int kThreads>
__device__ __forceinline__ void scan(const typename Elem<DT>::raw* __restrict__ x, int j1, Stat& st, Best& best) {
  constexpr int kTile = kThreads * kPer;
  typedef typename Elem<DT>::raw raw;
  constexpr int V = VEC ? 16 / (int)sizeof(raw) : 1;  // logits of a load
  const int tid = threadIdx.x;
  st = Stat{-INFINITY, 0.f, 0.f};
  for (int t0 = 0; t0 < j1; t0 += kTile) {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer / V; ++i) {
      const int j = t0 + (i * kThreads + tid) * V;
      if constexpr (VEC) {
        uint4 r = {0, 0, 0, 0};
        if (j + V <= j1) {
          r = *reinterpret_cast<const uint4*>(x + j);
          const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int e = 0; e < V; ++e) {
            if constexpr (DT == CL_F32)
              v[i * V + e] = __builtin_bit_cast(float, w[e]);
            else
              v[i * V + e] = Elem<DT>::up((uint16_t)(w[e / 2] >> (16 * (e % 2))));
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) v[i * V + e] = j + e < j1 ? Elem<DT>::up(x[j + e]) : -INFINITY;
        }
      } else {
        v[i] = j < j1 ? Elem<DT>::up(x[j]) : -INFINITY;
      }
    }
    float top = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) top = fmaxf(top, v[i]);
    // sums
    const float m = fmaxf(st.m, top);
    join(st, Stat{m, 0.f, 0.f});
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, w = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float d = v[i] - ref, e = __builtin_amdgcn_exp2f(d * kLog2e);
      l += e;
      w += fmaxf(d, -1000.f) * e;  // -inf adds nothing
    }
    st.l += l;
    st.w += w;
    // alternatives
    if (best.k) {
      float bar = best.bar;
      if (__builtin_popcountll(__ballot(top > bar)) > best.k) {
        // the k-th largest of the lanes' maxima, found from its highest bit down
        uint32_t u = __builtin_bit_cast(uint32_t, top + 0.0f), at_least = 0;
        u = top != top ? 0u : (u >> 31) ? ~u : u | 0x80000000u;
        for (int bit = 31; bit >= 0; --bit) {
          const uint32_t to = at_least | 1u << bit;
          if (__builtin_popcountll(__ballot(u >= to)) >= best.k) at_least = to;
        }
        bar = fmaxf(bar, key_value((u64)at_least << 32));
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const u64 who = __ballot(!(v[i] < bar));  // a NaN passes
        if (who) {
          const int j = t0 + (i / V * kThreads + tid) * V + i % V;
          best.insert(rank_key(v[i], j), who & __ballot(j < j1));
          bar = fmaxf(bar, best.bar);
        }
      }
    }
  }
}

// Joins the workgroup's wavefronts; the result is in wavefront 0 (st in all its lanes).
template <int kLpWaves>
__device__ __forceinline__ void join_waves(Stat& st, Best& best) {
  __shared__ float s_st[kLpWaves][3];
  __shared__ u64 s_top[kLpWaves][32];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  join_lanes(st);
  if (lane == 0) s_st[wave][0] = st.m, s_st[wave][1] = st.l, s_st[wave][2] = st.w;
  if (lane < best.k) s_top[wave][lane] = best.key;
  __syncthreads();
  if (wave) return;
  // the wavefronts' sums one to a lane, then their keys 64 at a time
  st = lane < kLpWaves ? Stat{s_st[lane][0], s_st[lane][1], s_st[lane][2]} : Stat{-INFINITY, 0.f, 0.f};
  join_lanes(st);
  const int keys = (kLpWaves - 1) * best.k;
  for (int k0 = 0; k0 < keys; k0 += 64) {
    const int i = k0 + lane;
    best.insert(i < keys ? s_top[1 + i / best.k][i % best.k] : 0, ~0ull);
  }
}

// A row's outputs, by wavefront 0.
template <int DT>
__device__ __forceinline__ void finish(const LogprobArgs& a, int t, const typename Elem<DT>::raw* x, const Stat& st,
                                       const Best& best) {
  const int lane = threadIdx.x % 64;
  const float lse = __builtin_amdgcn_logf(st.l) * kLn2;
  if (lane == 0) a.entropy[t] = lse - st.w / st.l;
  for (int c = lane; c < a.given; c += 64) {
    const int id = a.ids[(int64_t)t * a.given + c];
    a.logp[(int64_t)t * a.given + c] = id >= 0 && id < a.vocab ? Elem<DT>::up(x[id]) - st.m - lse : __builtin_nanf("");
  }
  if (lane < a.top_k) {
    const int id = (int)~(uint32_t)best.key;
    a.top_ids[(int64_t)t * a.top_k + lane] = id;
    a.top_logp[(int64_t)t * a.top_k + lane] = key_value(best.key) - st.m - lse;
  }
}

// One workgroup a row.
template <int DT, bool VEC, int kThreads>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobArgs a) {
  const int t = blockIdx.x;
  const auto* x = static_cast<const typename Elem<DT>::raw*>(a.x) + t * a.x_row;
  Stat st;
  Best best;
  best.clear(a.top_k);
  scan<DT, VEC, kThreads>(x, a.vocab, st, best);
  join_waves<kThreads / 64>(st, best);
  if (threadIdx.x < 64) finish<DT>(a, t, x, st, best);
}

template <int DT, int kThreads>
void launch_logprobs(const LogprobArgs& a, int rows, bool vec, hipStream_t s) {
  if (vec)
    hipLaunchKernelGGL((logprobs_kernel<DT, true, kThreads>), dim3(rows), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((logprobs_kernel<DT, false, kThreads>), dim3(rows), dim3(kThreads), 0, s, a);
}

template <int DT>
void launch_logprobs(const LogprobArgs& a, int rows, bool vec, hipStream_t s) {
  // four wavefronts a row where the rows fill the card, sixteen where they do not
  if (rows >= 512)
    launch_logprobs<DT, 256>(a, rows, vec, s);
  else
    launch_logprobs<DT, 1024>(a, rows, vec, s);
}

}  // namespace
}  // namespace cl

using namespace cl;

extern "C" cl_status cl_token_logprobs(const void* x, int32_t dtype, int64_t x_row, int32_t rows, int32_t vocab,
                                       const int32_t* ids, int32_t given, float* logp, float* entropy, int32_t top_k,
                                       int32_t* top_ids, float* top_logp, void* stream) {
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
  const LogprobArgs a = {x, x_row, ids, logp, entropy, top_ids, top_logp, vocab, given, top_k};
  // 16-byte loads where every row starts on a 16-byte boundary
  const bool vec = aligned_to(x, 16) && (x_row * (int64_t)elem_size(dtype)) % 16 == 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == CL_F16)
    launch_logprobs<CL_F16>(a, rows, vec, s);
  else if (dtype == CL_BF16)
    launch_logprobs<CL_BF16>(a, rows, vec, s);
  else
    launch_logprobs<CL_F32>(a, rows, vec, s);
  return launched("logprobs");
}
