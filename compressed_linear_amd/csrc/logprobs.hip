// logprobs.hip -- log probabilities of given tokens, entropy and top
// alternatives of each row of logits.
//
// One pass over a row: a thread takes 32 logits at a time into registers and
// keeps the running maximum m, l = sum exp(x - m) and w = sum (x - m) exp(x - m)
// of what it has seen (moving m by d turns w into (w - d l) e^-d, l into
// l e^-d); threads and wavefronts are joined by the same rule.  log p(i) = x_i - m - log l; entropy = log l - w / l.
//
// Alternatives: logits become 64-bit keys (order of the value, then of the lower id).
// With k wanted of W wavefronts, each wavefront names the ceil(k / W)-th largest of its lanes' maxima, and the
// ceil(k / that)-th largest of those is a bar that k logits reach.  What is below the bar, or below a wavefront's own one
// in a later tile, is none of the k, which one vote for most tiles, one for each four logits of a lane and one for each
// logit settle.  The few that pass are collected in LDS; a wavefront whose list is full
// keeps its best k, whose last then is an exact bar (rows of equal or mostly masked
// logits).  At the end the candidates above the highest bar of the workgroup are ranked by
// counting the larger ones: keys are unique, so a rank is a place in the output.
//
// Bound by the read of the logits where there are rows for the whole card (4096 rows of
// 32000 fp32 logits with 4 given tokens and 5 alternatives: 94 us, 5.6 TB/s); a single
// row by the latency of loads, votes and joins (32000 logits, 8 alternatives: 6.4 us, without alternatives 4.9; spread
// over eight workgroups that meet at a counter it took a microsecond more).
#include <type_traits>

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
// Running maximum and sums of some logits.
struct Stat {
  float m, l, w;
};
__device__ __forceinline__ void join(Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  // a side without a logit above -inf has l = w = 0 and adds nothing; nor does one far below, whose d times l may be past fp32 (a
  // row masked with the type's lowest value), so d is not taken below -1000 there, where e^d is 0
  const float da = a.m == m ? 0.f : a.m - m, db = b.m == m ? 0.f : b.m - m;
  const float ea = __builtin_amdgcn_exp2f(da * kLog2e), eb = __builtin_amdgcn_exp2f(db * kLog2e);
  a.w = ea * (a.w + fmaxf(da, -1000.f) * a.l) + eb * (b.w + fmaxf(db, -1000.f) * b.l);
  a.l = ea * a.l + eb * b.l;
  a.m = m;
}

// Reductions over a wavefront by lane permutes (rows of 16 lanes, then the four rows); every lane gets the same bits.
template <int CTRL>
__device__ __forceinline__ uint32_t permuted(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}
template <typename F>
__device__ __forceinline__ uint32_t reduced(uint32_t v, F f) {
  v = f(v, permuted<0xB1>(v));   // quad_perm [1,0,3,2]
  v = f(v, permuted<0x4E>(v));   // quad_perm [2,3,0,1]
  v = f(v, permuted<0x141>(v));  // row_half_mirror
  v = f(v, permuted<0x140>(v));  // row_mirror
  const auto row = [&](int r) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * r); };
  return f(f(row(0), row(1)), f(row(2), row(3)));
}
__device__ __forceinline__ float max_of_lanes(float v) {
  const auto f = [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
  };
  return __builtin_bit_cast(float, reduced(__builtin_bit_cast(uint32_t, v), f));
}
__device__ __forceinline__ float sum_of_lanes(float v) {
  const auto f = [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  };
  return __builtin_bit_cast(float, reduced(__builtin_bit_cast(uint32_t, v), f));
}
__device__ __forceinline__ void join_lanes(Stat& a) {
  join(a, Stat{max_of_lanes(a.m), 0.f, 0.f});
  a.l = sum_of_lanes(a.l);
  a.w = sum_of_lanes(a.w);
}

constexpr int kList = 128;  // candidates of a wavefront

// Keys of `list` larger than `key`.
__device__ __forceinline__ int rank_in(const u64* list, int n, u64 key) {
  int r = 0;
#pragma unroll 8
  for (int i = 0; i < n; ++i) r += list[i] > key;
  return r;
}

// A wavefront's candidates (uniform but for the list in LDS).
struct Best {
  u64* list;
  int k, n;
  float bar;  // what a logit must not be below
  u64 last;   // what a key has to beat; 0 until the list was full
  __device__ __forceinline__ void clear(u64* l, int top_k) {
    list = l;
    k = top_k;
    n = 0;
    bar = -INFINITY;
    last = 0;
  }
  // Keeps the best k.
  __device__ __forceinline__ void shrink() {
    const int lane = threadIdx.x % 64;
    lds_ordered();
    u64 key[kList / 64];
    int at[kList / 64];
#pragma unroll
    for (int i = 0; i < kList / 64; ++i) {
      key[i] = lane + 64 * i < n ? list[lane + 64 * i] : 0;
      at[i] = rank_in(list, n, key[i]);
    }
    lds_ordered();
#pragma unroll
    for (int i = 0; i < kList / 64; ++i)
      if (key[i] && at[i] < k) list[at[i]] = key[i];
    lds_ordered();
    n = min(n, k);
    if (n == k) {
      last = list[k - 1];
      last = (u64)(uint32_t)__builtin_amdgcn_readfirstlane((int)(last >> 32)) << 32 |
             (uint32_t)__builtin_amdgcn_readfirstlane((int)last);
      const float v = key_value(last);
      bar = fmaxf(bar, v != v ? INFINITY : v);  // a NaN is the last: only another NaN may pass
    }
  }
  // Adds the keys of the lanes in `who`.
  __device__ __forceinline__ void add(u64 key, u64 who) {
    if (last) who &= __ballot(key > last);
    if (n + __builtin_popcountll(who) > kList) {
      shrink();
      who &= __ballot(key > last);
    }
    const int lane = threadIdx.x % 64;
    if ((who >> lane) & 1) list[n + __builtin_popcountll(who & ((1ull << lane) - 1))] = key;
    n += __builtin_popcountll(who);
  }
  // The order of LDS accesses within the wavefront is theirs in the program.
  static __device__ __forceinline__ void lds_ordered() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }
};

// The n-th largest of the lanes' `u`, rounded down to its upper half, found from the highest bit down.
__device__ __forceinline__ uint32_t nth_of_lanes(uint32_t u, int n) {
  if (n == 1) return reduced(u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
  uint32_t at_least = 0;
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t to = at_least | 1u << bit;
    if (__builtin_popcountll(__ballot(u >= to)) >= n) at_least = to;
  }
  return at_least;
}

// A row's logits [0, n), by a workgroup of kThreads, from the 16-byte boundary at or before its start.
template <int DT, int kThreads>
__device__ __forceinline__ void scan(const typename Elem<DT>::raw* __restrict__ x, int n, Stat& st, Best& best) {
  typedef typename Elem<DT>::raw raw;
  constexpr int kTile = kThreads * kPer, kWaves = kThreads / 64;
  constexpr int V = 16 / (int)sizeof(raw);  // logits of a load
  __shared__ uint32_t s_bar[kWaves];
  const int tid = threadIdx.x, before = (int)(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(raw));
  st = Stat{-INFINITY, 0.f, 0.f};
  for (int t0 = -before; t0 < n; t0 += kTile) {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer / V; ++i) {
      const int j = t0 + (i * kThreads + tid) * V;
      if (j >= 0 && j + V <= n) {
        const uint4 r = *reinterpret_cast<const uint4*>(x + j);
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
        for (int e = 0; e < V; ++e) v[i * V + e] = -INFINITY;
        if (j < n) {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (j + e >= 0 && j + e < n) v[i * V + e] = Elem<DT>::up(x[j + e]);
        }
      }
    }
    constexpr int kGroup = 4, kGroups = kPer / kGroup;
    float g[kGroups], peak, top;  // largest of each four and of all, a NaN if there is one; largest without the fours that have one
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      g[i] = __builtin_elementwise_maximum(__builtin_elementwise_maximum(v[kGroup * i], v[kGroup * i + 1]),
                                           __builtin_elementwise_maximum(v[kGroup * i + 2], v[kGroup * i + 3]));
      peak = i ? __builtin_elementwise_maximum(peak, g[i]) : g[i];
      top = i ? fmaxf(top, g[i]) : g[i];
    }
    // sums
    const float m = fmaxf(st.m, top);
    join(st, Stat{m, 0.f, 0.f});
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, w = 0.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if (t0 + p * (kTile / 4) >= n) break;  // the rest of a row's last tile is empty
#pragma unroll
      for (int i = p * (kPer / 4); i < (p + 1) * (kPer / 4); ++i) {
        const float d = v[i] - ref, e = __builtin_amdgcn_exp2f(d * kLog2e);
        l += e;
        w += fmaxf(d, -1000.f) * e;  // -inf adds nothing
      }
    }
    st.l += l;
    st.w += w;
    // alternatives
    if (best.k) {
      uint32_t u = __builtin_bit_cast(uint32_t, top + 0.0f);
      u = top != top ? 0u : (u >> 31) ? ~u : u | 0x80000000u;
      if (t0 <= 0) {
        // where `enough` wavefronts have `each` lanes whose maxima reach a value, top_k logits do: the value is the enough-th
        // largest of their each-th largest
        const int each = (best.k + kWaves - 1) / kWaves, enough = (best.k + each - 1) / each;
        const uint32_t own = nth_of_lanes(u, each);
        if (tid % 64 == 0) s_bar[tid / 64] = own;
        __syncthreads();
        const uint32_t mine = s_bar[tid % kWaves];
        int reach = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) reach += s_bar[i] >= mine;
        best.bar = fmaxf(best.bar, key_value((u64)nth_of_lanes(reach >= enough ? mine : 0, 1) << 32));
      }
      if (__builtin_popcountll(__ballot(top > best.bar)) > best.k)
        best.bar = fmaxf(best.bar, key_value((u64)nth_of_lanes(u, best.k) << 32));
      if (!__any(!(peak < best.bar))) continue;
#pragma unroll
      for (int f = 0; f < kGroups; ++f) {
        if (!__any(!(g[f] < best.bar))) continue;
#pragma unroll
        for (int i = kGroup * f; i < kGroup * f + kGroup; ++i) {
          const u64 who = __ballot(!(v[i] < best.bar));  // a NaN passes
          if (who) {
            const int j = t0 + (i / V * kThreads + tid) * V + i % V;
            best.add(rank_key(v[i], j), who & __ballot(j >= 0 && j < n));
          }
        }
      }
    }
  }
}

// Joins the wavefronts' sums.
template <int kWaves>
__device__ __forceinline__ void join_waves(Stat& st) {
  __shared__ float s_st[kWaves][3];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  join_lanes(st);
  if (lane == 0) s_st[wave][0] = st.m, s_st[wave][1] = st.l, s_st[wave][2] = st.w;
  __syncthreads();
  st = lane < kWaves ? Stat{s_st[lane][0], s_st[lane][1], s_st[lane][2]} : Stat{-INFINITY, 0.f, 0.f};
  join_lanes(st);
}

// One workgroup a row.
template <int DT, int kThreads>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobArgs a) {
  constexpr int kWaves = kThreads / 64;
  __shared__ u64 s_list[kWaves * kList], s_all[kWaves * kList];
  __shared__ float s_bar[kWaves];
  __shared__ int s_n;
  const int t = blockIdx.x, tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const auto* x = static_cast<const typename Elem<DT>::raw*>(a.x) + t * a.x_row;
  const int first = tid < a.given ? a.ids[(int64_t)t * a.given + tid] : -1;
  if (tid == 0) s_n = 0;
  Stat st;
  Best best;
  best.clear(s_list + wave * kList, a.top_k);
  scan<DT, kThreads>(x, a.vocab, st, best);
  // the first given tokens' logits fly while the sums are joined
  float mine = __builtin_nanf("");
  if (first >= 0 && first < a.vocab) mine = Elem<DT>::up(x[first]);
  if (lane == 0) s_bar[wave] = best.bar;
  join_waves<kWaves>(st);  // a barrier: bars and the cleared count are there
  const float lse = __builtin_amdgcn_logf(st.l) * kLn2;
  if (tid == 0) a.entropy[t] = lse - st.w / st.l;
  for (int c = tid; c < a.given; c += kThreads) {
    if (c >= kThreads) {
      const int id = a.ids[(int64_t)t * a.given + c];
      mine = id >= 0 && id < a.vocab ? Elem<DT>::up(x[id]) : __builtin_nanf("");
    }
    a.logp[(int64_t)t * a.given + c] = mine - st.m - lse;
  }
  if (!a.top_k) return;
  // candidates above every wavefront's bar
  float bar = s_bar[0];
#pragma unroll
  for (int v = 1; v < kWaves; ++v) bar = fmaxf(bar, s_bar[v]);
  for (int i = lane; i < best.n; i += 64) {
    const u64 key = best.list[i];
    if (!(key_value(key) < bar)) s_all[atomicAdd(&s_n, 1)] = key;
  }
  __syncthreads();
  const int n = s_n;
  for (int i = tid; i < n; i += kThreads) {
    const u64 key = s_all[i];
    const int at = rank_in(s_all, n, key);
    if (at < a.top_k) {
      a.top_ids[(int64_t)t * a.top_k + at] = (int)~(uint32_t)key;
      a.top_logp[(int64_t)t * a.top_k + at] = key_value(key) - st.m - lse;
    }
  }
}

template <int DT>
void launch_logprobs(const LogprobArgs& a, int rows, hipStream_t s) {
  const auto go = [&](auto threads) {
    constexpr int n = decltype(threads)::value;
    in_pieces(rows, n, [&](int64_t first, int64_t count) {
      LogprobArgs b = a;
      b.x = beyond(a.x, DT, first * a.x_row);
      if (a.given) b.ids += first * a.given, b.logp += first * a.given;
      b.entropy += first;
      if (a.top_k) b.top_ids += first * a.top_k, b.top_logp += first * a.top_k;
      hipLaunchKernelGGL((logprobs_kernel<DT, n>), dim3((unsigned)count), dim3(n), 0, s, b);
    });
  };
  // As few wavefronts a row as hold it in one tile where rows abound, since a tile costs the same half empty (2048 logits, 4096
  // rows: 12 us with one, 26 with four), but four for few rows (2000 logits, one row, 32 alternatives: 6.8; 12.5 with one); four
  // too where rows abound (32000, 4096 rows: 98; 100 with eight, 142 with sixteen).  More while rows leave CUs free or are
  // long: sixteen for up to 256 rows (32000: 12.0; 13.1 with eight, 17.6 with four) unless eight hold the row (12000: 7.8; 8.8
  // with sixteen) and for long ones (151937, 1024 rows: 120; 131, 144), eight between (32000, 512 rows: 16.7; 20.6 with
  // four, 20.7 with sixteen).
  if (rows > 256 && a.vocab <= 64 * kPer)
    go(std::integral_constant<int, 64>());
  else if (rows > 256 && a.vocab <= 128 * kPer)
    go(std::integral_constant<int, 128>());
  else if (a.vocab <= 256 * kPer)
    go(std::integral_constant<int, 256>());
  else if (rows <= 256 ? a.vocab > 512 * kPer : a.vocab > 65536)
    go(std::integral_constant<int, 1024>());
  else if (rows <= 512)
    go(std::integral_constant<int, 512>());
  else
    go(std::integral_constant<int, 256>());
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
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == CL_F16)
    launch_logprobs<CL_F16>(a, rows, s);
  else if (dtype == CL_BF16)
    launch_logprobs<CL_BF16>(a, rows, s);
  else
    launch_logprobs<CL_F32>(a, rows, s);
  return launched("logprobs");
}
