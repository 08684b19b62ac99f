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
// Bound by the read of the logits.
#include "serving.h"

namespace cl {
namespace {

constexpr int kThreads = 256, kLpWaves = kThreads / 64;
constexpr int kPer = 32;                  // logits of a thread's tile
constexpr int kTile = kThreads * kPer;    // logits of a workgroup's tile
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
  float4* part;   // [rows, parts] (m, l, w, -)
  u64* part_top;  // [rows, parts, top_k]
  int vocab, given, top_k, parts, span;  // span: logits of a part
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

// One part of a row: its logits [j0, j1).
template <int DT, bool VEC>
__device__ __forceinline__ void scan(const typename Elem<DT>::raw* __restrict__ x, int j0, int j1, Stat& st, Best& best) {
  typedef typename Elem<DT>::raw raw;
  constexpr int V = VEC ? 16 / (int)sizeof(raw) : 1;  // logits of a load
  const int tid = threadIdx.x;
  st = Stat{-INFINITY, 0.f, 0.f};
  for (int t0 = j0; t0 < j1; t0 += kTile) {
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
__device__ __forceinline__ void join_waves(Stat& st, Best& best) {
  __shared__ float s_st[kLpWaves][3];
  __shared__ u64 s_top[kLpWaves][32];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  join_lanes(st);
  if (lane == 0) s_st[wave][0] = st.m, s_st[wave][1] = st.l, s_st[wave][2] = st.w;
  if (lane < best.k) s_top[wave][lane] = best.key;
  __syncthreads();
  if (wave) return;
  for (int v = 1; v < kLpWaves; ++v) {
    join(st, Stat{s_st[v][0], s_st[v][1], s_st[v][2]});
    if (best.k) best.insert(lane < best.k ? s_top[v][lane] : 0, best.k == 64 ? ~0ull : (1ull << best.k) - 1);
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

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobArgs a) {
  const int part = blockIdx.x % a.parts, t = blockIdx.x / a.parts;
  const auto* x = static_cast<const typename Elem<DT>::raw*>(a.x) + t * a.x_row;
  Stat st;
  Best best;
  best.clear(a.top_k);
  const int j0 = part * a.span;
  scan<DT, VEC>(x, j0, min(j0 + a.span, a.vocab), st, best);
  join_waves(st, best);
  if (threadIdx.x >= 64) return;
  if (a.parts == 1) {
    finish<DT>(a, t, x, st, best);
  } else {
    if (threadIdx.x == 0) a.part[blockIdx.x] = make_float4(st.m, st.l, st.w, 0.f);
    if ((int)threadIdx.x < a.top_k) a.part_top[(int64_t)blockIdx.x * a.top_k + threadIdx.x] = best.key;
  }
}

// Joins a row's parts: one wavefront a row.
template <int DT>
__global__ void __launch_bounds__(64) logprobs_join_kernel(LogprobArgs a) {
  const int t = blockIdx.x, lane = threadIdx.x;
  Stat st = {-INFINITY, 0.f, 0.f};
  Best best;
  best.clear(a.top_k);
  for (int p = lane; p < a.parts; p += 64) {
    const float4 v = a.part[(int64_t)t * a.parts + p];
    join(st, Stat{v.x, v.y, v.z});
  }
  join_lanes(st);
  const int keys = a.parts * a.top_k;
  for (int k0 = 0; k0 < keys; k0 += 64) {
    const int k = k0 + lane;
    best.insert(k < keys ? a.part_top[(int64_t)t * keys + k] : 0, ~0ull);
  }
  finish<DT>(a, t, static_cast<const typename Elem<DT>::raw*>(a.x) + t * a.x_row, st, best);
}

// Parts of a row: one where the rows fill the card, otherwise parts of at least 2048 logits.
struct LogprobPlan {
  int parts, span;
  size_t stat_bytes, need;
};
LogprobPlan plan_logprobs(int64_t rows, int vocab, int top_k) {
  LogprobPlan p;
  int64_t parts = (1024 + rows - 1) / rows;
  const int64_t most = (vocab + 2047) / 2048;
  if (rows >= 512) parts = 1;
  if (parts > most) parts = most;
  p.span = (int)((vocab + parts - 1) / parts + 15) / 16 * 16;
  p.parts = (vocab + p.span - 1) / p.span;
  p.stat_bytes = p.parts > 1 ? (size_t)rows * p.parts * sizeof(float4) : 0;
  p.need = p.parts > 1 ? p.stat_bytes + (size_t)rows * p.parts * top_k * sizeof(u64) : 0;
  return p;
}

template <int DT>
void launch_logprobs(const LogprobArgs& a, int rows, bool vec, hipStream_t s) {
  const dim3 grid((unsigned)rows * a.parts);
  if (vec)
    hipLaunchKernelGGL((logprobs_kernel<DT, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((logprobs_kernel<DT, false>), grid, dim3(kThreads), 0, s, a);
  if (a.parts > 1) hipLaunchKernelGGL((logprobs_join_kernel<DT>), dim3(rows), dim3(64), 0, s, a);
}

}  // namespace
}  // namespace cl

using namespace cl;

extern "C" size_t cl_token_logprobs_work_bytes(int32_t rows, int32_t vocab, int32_t top_k) {
  if (rows < 1 || vocab < 1 || top_k < 0) return 0;
  return plan_logprobs(rows, vocab, top_k).need;
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
  const LogprobPlan p = plan_logprobs(rows, vocab, top_k);
  if ((int64_t)rows * p.parts > 0x7FFFFFFF) return fail(CL_ESIZE, "logprobs: too many rows");
  if (p.need && (!work || work_bytes < p.need))
    return fail(CL_ENOMEM, "logprobs: work has %zu bytes, %zu are needed", work_bytes, p.need);
  if (!aligned_to(work, 16)) return fail(CL_EINVAL, "logprobs: work must be 16-byte aligned");
  const LogprobArgs a = {x, x_row, ids, logp, entropy, top_ids, top_logp, static_cast<float4*>(work),
                         reinterpret_cast<u64*>(static_cast<uint8_t*>(work) + p.stat_bytes), vocab, given, top_k, p.parts,
                         p.span};
  // 16-byte loads where every row starts on a 16-byte boundary (parts do, as spans are multiples of 16)
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
