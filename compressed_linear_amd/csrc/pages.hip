// pages.hip -- the pages of caches: which sequence holds which (given out, forked, taken back, compacted), and the
// moves inside a cache that follow from it (whole pages, accepted drafts).
#include <algorithm>

#include "serving.h"

namespace cl {
namespace {

constexpr int kMostSequences = 4096;
constexpr int kMostKept = 256;
constexpr int kScan = 16384;  // pages that a workgroup looks at together, 16 to a thread

struct Pool {
  int32_t *table, *lens, *refs, *left_out;
  int sequences, width, pages, page_shift;
  __device__ __forceinline__ bool has(int page) const { return page >= 0 && page < pages; }
  __device__ __forceinline__ int held(int tokens) const { return (tokens + (1 << page_shift) - 1) >> page_shift; }
};

// Sum of v over the threads before this one of a workgroup of 1024, and over all of them.
struct Before {
  int before, all;
};
__device__ __forceinline__ Before sum_before(int v, int* waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int up = __shfl_up(s, d);
    if (lane >= d) s += up;
  }
  if (lane == 63) waves[wave] = s;
  __syncthreads();
  int before = s - v, all = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    const int n = waves[w];
    before += w < wave ? n : 0;
    all += n;
  }
  __syncthreads();
  return {before, all};
}

// 16 pages from `first` on as bits: free ones (refs 0) where FREE, held ones otherwise; none past `end`.
template <bool FREE>
__device__ __forceinline__ uint32_t sixteen(const int32_t* refs, int first, int end) {
  uint32_t bits = 0;
  if (first + 16 <= end && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
    const w4* p = reinterpret_cast<const w4*>(refs + first);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const w4 v = p[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) bits |= (uint32_t)((v[j] == 0) == FREE) << (4 * i + j);
    }
  } else {
    for (int i = 0; i < 16 && first + i < end; ++i) bits |= (uint32_t)((refs[first + i] == 0) == FREE) << i;
  }
  return bits;
}

// Each number of the n in `base` replaced by the largest up to it, by a workgroup of `THREADS`.
template <int THREADS>
__device__ __forceinline__ void running_max(int* base, int n, int* waves) {
  const int per = (n + THREADS - 1) / THREADS, first = min(per * (int)threadIdx.x, n), end = min(first + per, n);
  int m = INT32_MIN;
  for (int i = first; i < end; ++i) base[i] = m = max(m, base[i]);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int up = __shfl_up(m, d);
    if (lane >= d) m = max(m, up);
  }
  if (lane == 63) waves[wave] = m;
  int before = __shfl_up(m, 1);
  if (lane == 0) before = INT32_MIN;
  __syncthreads();
  for (int w = 0; w < wave; ++w) before = max(before, waves[w]);
  for (int i = first; i < end; ++i) base[i] = max(base[i], before);
  __syncthreads();
}

// The last of n numbers in order that is at most t, the first if none is.
__device__ __forceinline__ int sequence_of(const int* base, int n, int t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (base[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------- extend
// One workgroup: every page that is given out depends on how many were before.  A thread has up to four sequences
// side by side, so that their order is the threads'.  Pages are found kScan at a time, lowest first, until there are enough; a free
// page's number among the free ones says whose it is, by a search in the sequences' ends.  Bound by the chain of loads: the
// sequences' tokens, their last pages, those pages' counts, the pages given, the slots (8.5 us for 64 sequences of 16 drafts; a scan past
// held pages is 1.8 us for each kScan of them).
__global__ void __launch_bounds__(1024) pool_extend_kernel(Pool p, const int32_t* __restrict__ cu, int tokens,
                                                           int32_t* __restrict__ slots, int32_t* __restrict__ src,
                                                           int32_t* __restrict__ dst, int inline_slots) {
  __shared__ __attribute__((aligned(16))) int last[kMostSequences];   // a sequence's last page where its tokens join it, -1
  __shared__ int ends[kMostSequences];   // pages given to it and those before
  __shared__ int from[kMostSequences];   // its first place that is given a page
  __shared__ int base[kMostSequences + 1];  // its first new token's number (cu), or the largest of those before
  __shared__ int list[kScan];            // free pages, a scan's
  __shared__ int waves[16];
  __shared__ int left;
  const int B = p.sequences, tid = threadIdx.x, page = 1 << p.page_shift, per = (B + 1023) / 1024;
  const auto sequence = [&](int i) { return i < per ? per * tid + i : B; };  // a thread's, B where it has none
  const uint32_t free0 = sixteen<true>(p.refs, 16 * tid, p.pages);  // asked for before anything is known, as are the next three
  int len[4], more[4], want[4], mine[4], holders[4];
  bool go[4], any[4];
  for (int b = tid; b <= B; b += 1024) base[b] = cu[b];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = sequence(i);
    len[i] = b < B ? p.lens[b] : -1;
    more[i] = b < B ? cu[b] : 0;
    want[i] = b < B ? cu[b + 1] : 0;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int place = len[i] >> p.page_shift;
    const bool part = len[i] > 0 && len[i] & (page - 1) && place < p.width;
    mine[i] = part ? p.table[(int64_t)sequence(i) * p.width + place] : -1;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) holders[i] = p.has(mine[i]) ? p.refs[mine[i]] : 0;
  if (tid == 0) left = 0;
  __syncthreads();
  running_max<1024>(base, B + 1, waves);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = sequence(i);
    const int a = more[i], z = want[i];
    any[i] = a != z;
    more[i] = want[i] = 0;
    go[i] = false;
    if (b >= B) continue;
    const bool fits = a >= 0 && a == base[b] && z >= a && z <= tokens;
    more[i] = fits ? z - a : 0;
    go[i] = more[i] > 0 && len[i] >= 0 && (int64_t)len[i] + more[i] <= (int64_t)p.width << p.page_shift;
    if (go[i] && (len[i] & (page - 1))) go[i] = p.has(mine[i]);
    if (!go[i]) mine[i] = -1;
    last[b] = mine[i];
    want[i] = go[i] ? p.held(len[i] + more[i]) - p.held(len[i]) : 0;
  }
  __syncthreads();
  // A last page that others hold too is copied, but for the last of its holders if all of them are extended: k extended
  // ones before leave refs - k holders.
  bool shared[4];
  int need = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = sequence(i);
    shared[i] = false;
    if (mine[i] >= 0) {
      if (holders[i] > 1) {
        int j = 0;
        for (; j + 4 <= b; j += 4) {
          const int4 v = *reinterpret_cast<const int4*>(last + j);
          holders[i] -= (v.x == mine[i]) + (v.y == mine[i]) + (v.z == mine[i]) + (v.w == mine[i]);
        }
        for (; j < b; ++j) holders[i] -= last[j] == mine[i];
      }
      shared[i] = holders[i] > 1;
    }
    want[i] += shared[i];
    need += want[i];
  }
  const Before all = sum_before(need, waves);
  int end = all.before;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = sequence(i);
    end += want[i];
    if (b < B) {
      ends[b] = end;
      from[b] = p.held(len[i]) - shared[i];
    }
  }
  __syncthreads();
  // Free pages, lowest first, into a list, and from there to places: each thread takes one at a time, whoever found it.
  int found = 0;
  for (int64_t first = 0; first < p.pages && found < all.all; first += kScan) {
    const int at = (int)min(first + 16 * tid, (int64_t)p.pages);
    uint32_t bits = first ? sixteen<true>(p.refs, at, p.pages) : free0;
    const Before rank = sum_before(__popc(bits), waves);
    for (int k = rank.before; bits && found + k < all.all; bits &= bits - 1, ++k) list[k] = at + __builtin_ctz(bits);
    __syncthreads();
    for (int k = found + tid; k < min(found + rank.all, all.all); k += 1024) {
      const int given = list[k - found];
      int lo = 0, hi = B - 1;  // the first sequence that ends past k
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (ends[mid] > k)
          hi = mid;
        else
          lo = mid + 1;
      }
      const int i = k - (lo ? ends[lo - 1] : 0);
      p.table[(int64_t)lo * p.width + from[lo] + i] = given;
      p.refs[given] = 1;
    }
    found += rank.all;
    __syncthreads();
  }
  found = min(found, all.all);
  // Whoever ends past the pages found is left out, and with it everyone after: what it was given goes back.
  int out = 0;
  end = all.before;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = sequence(i);
    if (b >= B) continue;
    const int start = end;
    end += want[i];
    int32_t* row = p.table + (int64_t)b * p.width;
    const bool served = go[i] && end <= found;
    int copied_from = -1, copied_to = -1;
    if (go[i] && !served) {
      const int place = from[b];
      for (int k = start; k < found; ++k) {
        p.refs[row[place + k - start]] = 0;
        row[place + k - start] = k == start && shared[i] ? mine[i] : -1;
      }
    }
    if (served && shared[i]) {
      copied_from = mine[i];
      copied_to = row[from[b]];
      atomicSub(&p.refs[mine[i]], 1);
    }
    src[b] = copied_from;
    dst[b] = copied_to;
    if (served)
      p.lens[b] = len[i] + more[i];
    else if (any[i])
      ++out;
    last[b] = served ? len[i] : -1;  // from here on: tokens before the new ones
  }
  if (out) atomicAdd(&left, out);
  __syncthreads();
  if (tid == 0) *p.left_out = left;
  const auto slot_of = [&](int t) {
    const int lo = sequence_of(base, B, t);
    if (t < base[lo] || t >= base[lo + 1] || last[lo] < 0) return -1;
    const int place = last[lo] + t - base[lo];
    return p.table[(int64_t)lo * p.width + (place >> p.page_shift)] << p.page_shift | (place & (page - 1));
  };
  if (inline_slots) {
    for (int t = tid; t < tokens; t += 1024) slots[t] = slot_of(t);
  } else {  // each sequence's first token, which says whether it was served
    for (int b = tid; b < B; b += 1024)
      if (base[b] >= 0 && base[b] < tokens && base[b + 1] > base[b]) slots[base[b]] = slot_of(base[b]);
  }
}

// Slots of many tokens, once the pages are given: a sequence's first one says whether it was served.
__global__ void __launch_bounds__(256) pool_slots_kernel(Pool p, const int32_t* __restrict__ cu, int tokens,
                                                         int32_t* __restrict__ slots) {
  __shared__ int base[kMostSequences + 1];
  __shared__ int waves[4];
  for (int b = threadIdx.x; b <= p.sequences; b += 256) base[b] = cu[b];
  __syncthreads();
  running_max<256>(base, p.sequences + 1, waves);
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= tokens) return;
  const int b = sequence_of(base, p.sequences, t), a = base[b], z = base[b + 1];
  if (t == a && z > a) return;
  int slot = -1;
  if (a >= 0 && t > a && t < z && slots[a] >= 0) {
    const int place = p.lens[b] - (z - t);
    slot = p.table[(int64_t)b * p.width + (place >> p.page_shift)] << p.page_shift | (place & ((1 << p.page_shift) - 1));
  }
  slots[t] = slot;
}

// --------------------------------------------------------------------- fork
// A workgroup has some places of all sequences: it reads them all before it writes any, so that sequences can take each
// other's rows.  Of all workgroups the first one has the lengths too; `block` are in launches before this one.  Bound by the chain of
// loads and the holders' counts (4.3 us for 64 sequences).
constexpr int kForkWords = 16384;
__global__ void __launch_bounds__(1024) pool_fork_kernel(Pool p, const int32_t* __restrict__ parents, int columns, int block) {
  __shared__ int old[kForkWords];
  block += blockIdx.x;
  const int B = p.sequences, first = block * columns, n = min(columns, p.width - first);
  for (int i = threadIdx.x; i < B * n; i += 1024) old[i] = p.table[(int64_t)(i / n) * p.width + first + i % n];
  int lens[kMostSequences / 1024];
#pragma unroll
  for (int i = 0; i < kMostSequences / 1024; ++i) {
    const int b = i * 1024 + threadIdx.x;
    if (block || b >= B) continue;
    const int from = parents[b];
    lens[i] = from >= 0 && from < B ? p.lens[from] : 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < B * n; i += 1024) {
    const int b = i / n, from = parents[b];
    const int was = old[i], now = from >= 0 && from < B ? old[from * n + i % n] : -1;
    if (was == now) continue;
    p.table[(int64_t)b * p.width + first + i % n] = now;
    if (p.has(was)) atomicSub(&p.refs[was], 1);
    if (p.has(now)) atomicAdd(&p.refs[now], 1);
  }
#pragma unroll
  for (int i = 0; i < kMostSequences / 1024; ++i) {
    const int b = i * 1024 + threadIdx.x;
    if (block == 0 && b < B) p.lens[b] = lens[i];
  }
}

// ----------------------------------------------------------------- truncate
// A wavefront a sequence, since a sequence mostly gives back few pages at a time.  Bound by the launch then (1.4 to 3 us); a long
// sequence's end is 64 pages at a time, one load after another (8192 pages 41 us).
__global__ void __launch_bounds__(64) pool_truncate_kernel(Pool p, const int32_t* __restrict__ to) {
  const int b = blockIdx.x, len = p.lens[b], n = to[b];
  if (n < 0 || n >= len) return;
  int32_t* row = p.table + (int64_t)b * p.width;
  for (int w = p.held(n) + threadIdx.x; w < p.width; w += 64) {
    const int page = row[w];
    if (page < 0) break;  // a sequence's pages come first, then none
    if (p.has(page)) atomicSub(&p.refs[page], 1);
    row[w] = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) p.lens[b] = n;
}

// ------------------------------------------------------------------ compact
// One workgroup.  With n pages held, those from n on move to the free ones below n: the highest to the lowest, up to
// `most` of them.  Both lists are found by scans, then a thread takes a move at a time.  work[page] is where a moved page went,
// work[pages] the lowest page that moved.  Bound by the scans and the moves' loads (9 us for 2948 moves); the table's new names
// are a launch of their own, all of its entries side by side (4.7 us).
__global__ void __launch_bounds__(1024) pool_compact_kernel(Pool p, int most, int32_t* __restrict__ src,
                                                            int32_t* __restrict__ dst, int32_t* __restrict__ work) {
  __shared__ int waves[16];
  const int tid = threadIdx.x;
  const uint32_t held0 = sixteen<false>(p.refs, 16 * tid, p.pages);
  const auto held_at = [&](int64_t first) { return first ? sixteen<false>(p.refs, (int)min(first + 16 * tid, (int64_t)p.pages), p.pages) : held0; };
  int held = 0;
  for (int64_t first = 0; first < p.pages; first += kScan) held += __popc(held_at(first));
  held = sum_before(held, waves).all;
  int holes = 0;
  for (int64_t first = 0; first < held; first += kScan) {
    const int at = (int)min(first + 16 * tid, (int64_t)held), n = min(16, held - at);
    uint32_t bits = n > 0 ? ~held_at(first) & (0xffffu >> (16 - n)) : 0;
    const Before rank = sum_before(__popc(bits), waves);
    for (int k = holes + rank.before; bits && k < most; bits &= bits - 1, ++k) dst[k] = at + __builtin_ctz(bits);
    holes += rank.all;
  }
  const int moves = min(holes, most);
  int before = 0;  // held pages from `held` on; there are as many as holes
  for (int64_t first = (int64_t)held / kScan * kScan; first < p.pages; first += kScan) {
    const int64_t at = first + 16 * tid;
    uint32_t bits = held_at(first);
    if (at < held) bits &= at + 16 <= held ? 0u : ~0u << (held - at);
    const Before rank = sum_before(__popc(bits), waves);
    for (int k = holes - 1 - before - rank.before; bits; bits &= bits - 1, --k)
      if (k < moves) src[k] = (int)at + __builtin_ctz(bits);
    before += rank.all;
  }
  __syncthreads();
  for (int k = tid; k < most; k += 1024) {
    if (k >= moves) {
      src[k] = dst[k] = -1;
      continue;
    }
    const int from = src[k], to = dst[k];
    work[from] = to;
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
    if (k == moves - 1) work[p.pages] = from;
  }
  if (tid == 0 && moves == 0) work[p.pages] = p.pages;
}

__global__ void __launch_bounds__(256) pool_rename_kernel(Pool p, const int32_t* __restrict__ work) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= (int64_t)p.sequences * p.width) return;
  const int page = p.table[at];
  if (page >= work[p.pages] && page < p.pages) p.table[at] = work[page];
}

// --------------------------------------------------------------- copy pages
// A page of a cache is four runs of bytes (codes and scales of K and V); a workgroup copies one piece of one of them, four loads of 16 bytes
// under way in a thread.  Bound by memory (2948 pages of 133 KB 141 to 155 us from card to card, 5.2 to 5.7 TB/s read and
// written).
struct CopyArgs {
  const int32_t *src, *dst;
  uint8_t* run[4];
  int64_t bytes[4];
  int pieces[4];  // a page's pieces up to and with this run
  int pages;
};
constexpr int kPiece = 16384;
__global__ void __launch_bounds__(256) kv_copy_pages_kernel(CopyArgs a) {
  const int from = a.src[blockIdx.y], to = a.dst[blockIdx.y];
  if (from < 0 || from >= a.pages || to < 0 || to >= a.pages || from == to) return;
  int r = 0;
  while (r < 3 && (int)blockIdx.x >= a.pieces[r]) ++r;
  const int64_t first = (int64_t)(blockIdx.x - (r ? a.pieces[r - 1] : 0)) * kPiece;
  const w4* x = reinterpret_cast<const w4*>(a.run[r] + from * a.bytes[r] + first);
  w4* y = reinterpret_cast<w4*>(a.run[r] + to * a.bytes[r] + first);
  const int64_t left = a.bytes[r] - first;
  w4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = i * 256 + threadIdx.x;
    if (16 * k < left) v[i] = x[k];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = i * 256 + threadIdx.x;
    if (16 * k < left) y[k] = v[i];
  }
}

// --------------------------------------------------------------------- keep
// A workgroup has the drafts of a sequence for one head, K or V: all are read before any is written, so a draft may move to
// another's place.  Rows are 16-byte pieces (int4 heads of 64 have two), HELD of them to a thread.
struct KeepArgs {
  cl_kv_cache c;
  const int32_t *table, *lens, *kept;
  int width, most, page_shift;
};
template <int HELD>
__global__ void __launch_bounds__(256) kv_keep_kernel(KeepArgs a) {
  const int b = blockIdx.x, h = blockIdx.y, which = blockIdx.z;
  const bool int8 = a.c.kind == CL_KV_INT8;
  const int units = int8 ? a.c.dim / 16 : a.c.dim / 32, scales = int8 ? 1 : a.c.dim / 32;
  const int64_t len = a.lens[b];
  // the row of a place, -1 where it is none
  const auto row_of = [&](int64_t place) -> int64_t {
    if (place < 0 || place >> a.page_shift >= a.width) return -1;
    const int page = a.table[(int64_t)b * a.width + (place >> a.page_shift)];
    if (page < 0 || page >= a.c.pages) return -1;
    return (((int64_t)page * a.c.heads + h) << a.page_shift) + (place & (a.c.page_size - 1));
  };
  const auto move_of = [&](int j, int64_t* from, int64_t* to) {
    const int i = a.kept[(int64_t)b * a.most + j];
    *from = *to = -1;
    if (i < 0 || i == j) return;
    *from = row_of(len + i);
    *to = row_of(len + j);
    if (*to < 0) *from = -1;
  };
  w4* codes = static_cast<w4*>(which ? a.c.v : a.c.k);
  uint16_t* scale = which ? a.c.v_scale : a.c.k_scale;
  w4 v[HELD];
  int64_t to[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    to[i] = -1;
    const int k = i * blockDim.x + threadIdx.x;
    if (k >= a.most * units) continue;
    int64_t from, row;
    move_of(k / units, &from, &row);
    if (from < 0) continue;
    to[i] = row * units + k % units;
    v[i] = codes[from * units + k % units];
  }
  uint16_t s[4];
  int64_t s_to = -1;
  if (threadIdx.x < a.most) {
    int64_t from, row;
    move_of(threadIdx.x, &from, &row);
    if (from >= 0) {
      s_to = row * scales;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < scales) s[i] = scale[from * scales + i];
    }
  }
  __builtin_amdgcn_s_waitcnt(0);  // every row is in registers before any place is written
  __syncthreads();
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (to[i] >= 0) codes[to[i]] = v[i];
  if (s_to >= 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < scales) scale[s_to + i] = s[i];
  }
}

cl_status check_pool(const cl_page_pool* p, Pool* out) {
  if (!p) return fail(CL_EINVAL, "pool is NULL");
  if (!p->block_table || !p->lens || !p->refs || !p->left_out) return fail(CL_EINVAL, "pool: a pointer is NULL");
  if (!aligned_to(p->block_table, 4) || !aligned_to(p->lens, 4) || !aligned_to(p->refs, 4) || !aligned_to(p->left_out, 4))
    return fail(CL_EINVAL, "pool: a pointer is misaligned");
  if (p->sequences < 1 || p->width < 1 || p->pages < 1) return fail(CL_EINVAL, "pool: sizes must be >= 1");
  if (p->page_size < 16 || p->page_size > 1024 || (p->page_size & (p->page_size - 1)))
    return fail(CL_EINVAL, "pool: page_size %d is no power of two in [16, 1024]", p->page_size);
  if (p->sequences > kMostSequences) return fail(CL_ESIZE, "pool: more than %d sequences", kMostSequences);
  if ((int64_t)p->pages * p->page_size >= ((int64_t)1 << 31) || (int64_t)p->width * p->page_size >= ((int64_t)1 << 31))
    return fail(CL_ESIZE, "pool: 2^31 slots or more");
  *out = Pool{p->block_table, p->lens, p->refs, p->left_out, p->sequences, p->width, p->pages, __builtin_ctz(p->page_size)};
  return CL_OK;
}

}  // namespace
}  // namespace cl

using namespace cl;

extern "C" cl_status cl_pool_extend(const cl_page_pool* pool, const int32_t* cu_q, int32_t tokens, int32_t* slots,
                                    int32_t* src, int32_t* dst, void* stream) {
  clear_error();
  Pool p;
  cl_status st = check_pool(pool, &p);
  if (st != CL_OK) return st;
  if (tokens < 0) return fail(CL_EINVAL, "extend: tokens must be >= 0");
  if (!cu_q || (tokens && !slots) || !src || !dst) return fail(CL_EINVAL, "extend: a required pointer is NULL");
  if (!aligned_to(cu_q, 4) || !aligned_to(slots, 4) || !aligned_to(src, 4) || !aligned_to(dst, 4))
    return fail(CL_EINVAL, "extend: a pointer is misaligned");
  const int here = tokens <= 4096;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(pool_extend_kernel, dim3(1), dim3(1024), 0, s, p, cu_q, tokens, slots, src, dst, here);
  if (!here) hipLaunchKernelGGL(pool_slots_kernel, dim3((unsigned)(((int64_t)tokens + 255) / 256)), dim3(256), 0, s, p, cu_q, tokens, slots);
  return launched("extend");
}

extern "C" cl_status cl_pool_fork(const cl_page_pool* pool, const int32_t* parents, void* stream) {
  clear_error();
  Pool p;
  cl_status st = check_pool(pool, &p);
  if (st != CL_OK) return st;
  if (!parents || !aligned_to(parents, 4)) return fail(CL_EINVAL, "fork: parents is NULL or misaligned");
  const int columns = std::min(16, kForkWords / p.sequences);
  // tables of 2^26 places and more have more threads than a launch
  in_pieces(((int64_t)p.width + columns - 1) / columns, 1024, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL(pool_fork_kernel, dim3((unsigned)count), dim3(1024), 0, static_cast<hipStream_t>(stream), p, parents, columns,
                       (int)first);
  });
  return launched("fork");
}

extern "C" cl_status cl_pool_truncate(const cl_page_pool* pool, const int32_t* lens, void* stream) {
  clear_error();
  Pool p;
  cl_status st = check_pool(pool, &p);
  if (st != CL_OK) return st;
  if (!lens || !aligned_to(lens, 4)) return fail(CL_EINVAL, "truncate: lens is NULL or misaligned");
  if (lens == pool->lens) return fail(CL_EINVAL, "truncate: lens are the pool's own");
  hipLaunchKernelGGL(pool_truncate_kernel, dim3((unsigned)p.sequences), dim3(64), 0, static_cast<hipStream_t>(stream), p, lens);
  return launched("truncate");
}

extern "C" size_t cl_pool_compact_work_bytes(int32_t pages) { return pages < 1 ? 0 : 4 * ((size_t)pages + 1); }

extern "C" cl_status cl_pool_compact(const cl_page_pool* pool, int32_t max_moves, int32_t* src, int32_t* dst, void* work,
                                     size_t work_bytes, void* stream) {
  clear_error();
  Pool p;
  cl_status st = check_pool(pool, &p);
  if (st != CL_OK) return st;
  if (max_moves < 0) return fail(CL_EINVAL, "compact: max_moves must be >= 0");
  if (max_moves == 0) return CL_OK;
  if (!src || !dst || !work) return fail(CL_EINVAL, "compact: a required pointer is NULL");
  if (!aligned_to(src, 4) || !aligned_to(dst, 4) || !aligned_to(work, 4)) return fail(CL_EINVAL, "compact: a pointer is misaligned");
  if (work_bytes < cl_pool_compact_work_bytes(p.pages)) return fail(CL_ENOMEM, "compact: the workspace is too small");
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(pool_compact_kernel, dim3(1), dim3(1024), 0, s, p, max_moves, src, dst, static_cast<int32_t*>(work));
  in_pieces((int64_t)p.sequences * p.width, 2, [&](int64_t first, int64_t count) {
    Pool q = p;  // the table's entries in one row, fewer than 2^31 at a time
    q.table += first;
    q.sequences = 1;
    q.width = (int)count;
    hipLaunchKernelGGL(pool_rename_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, s, q, static_cast<const int32_t*>(work));
  });
  return launched("compact");
}

extern "C" cl_status cl_kv_copy_pages(const cl_kv_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                                      void* stream) {
  clear_error();
  cl_status st = check_cache(cache);
  if (st != CL_OK) return st;
  if (n < 0) return fail(CL_EINVAL, "copy pages: n must be >= 0");
  if (n == 0) return CL_OK;
  if (!src || !dst || !aligned_to(src, 4) || !aligned_to(dst, 4))
    return fail(CL_EINVAL, "copy pages: src or dst is NULL or misaligned");
  if (!aligned_to(cache->k_scale, 16) || !aligned_to(cache->v_scale, 16))
    return fail(CL_EINVAL, "copy pages: scales must be 16-byte aligned");
  const int64_t rows = (int64_t)cache->heads * cache->page_size;
  const int64_t codes = rows * (cache->kind == CL_KV_INT8 ? cache->dim : cache->dim / 2);
  const int64_t scales = rows * 2 * (cache->kind == CL_KV_INT8 ? 1 : cache->dim / 32);
  CopyArgs a = {src, dst, {static_cast<uint8_t*>(cache->k), static_cast<uint8_t*>(cache->v), reinterpret_cast<uint8_t*>(cache->k_scale),
                reinterpret_cast<uint8_t*>(cache->v_scale)}, {codes, codes, scales, scales}, {}, cache->pages};
  int64_t pieces = 0;
  for (int r = 0; r < 4; ++r) a.pieces[r] = (int)(pieces += (a.bytes[r] + kPiece - 1) / kPiece);
  hipStream_t s = static_cast<hipStream_t>(stream);
  for (int64_t first = 0; first < n; first += 65535) {
    CopyArgs b = a;
    b.src += first;
    b.dst += first;
    hipLaunchKernelGGL(kv_copy_pages_kernel, dim3((unsigned)pieces, (unsigned)std::min<int64_t>(65535, n - first)), dim3(256), 0, s, b);
  }
  return launched("copy pages");
}

extern "C" cl_status cl_kv_keep(const cl_kv_cache* cache, const int32_t* block_table, int32_t table_width,
                                int32_t sequences, const int32_t* ctx_lens, const int32_t* kept, int32_t most,
                                void* stream) {
  clear_error();
  cl_status st = check_cache(cache);
  if (st != CL_OK) return st;
  if (sequences < 0 || table_width < 1 || most < 0) return fail(CL_EINVAL, "keep: sequences, most >= 0 and table_width >= 1 are wanted");
  if (most > kMostKept) return fail(CL_EUNSUPPORTED, "keep: more than %d entries to a sequence", kMostKept);
  if (sequences == 0 || most == 0) return CL_OK;
  if (!block_table || !ctx_lens || !kept) return fail(CL_EINVAL, "keep: a required pointer is NULL");
  if (!aligned_to(block_table, 4) || !aligned_to(ctx_lens, 4) || !aligned_to(kept, 4))
    return fail(CL_EINVAL, "keep: a pointer is misaligned");
  if (sequences > 65535) return fail(CL_ESIZE, "keep: more than 65535 sequences");
  const KeepArgs a = {*cache, block_table, ctx_lens, kept, table_width, most, __builtin_ctz(cache->page_size)};
  // as few threads as have a piece each, since more only pass through (64 sequences x 8 heads of 8 drafts 3.2 us with 64 threads, 3.3 with
  // 256); two pieces a thread cost more (16 drafts 3.8 us with 64 threads, 3.3 with 128)
  const int pieces = most * (cache->kind == CL_KV_INT8 ? cache->dim / 16 : cache->dim / 32), threads = std::min(256, (pieces + 63) / 64 * 64);
  const auto kernel = pieces <= 256 ? kv_keep_kernel<1> : pieces <= 512 ? kv_keep_kernel<2> : kv_keep_kernel<8>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)sequences, (unsigned)cache->heads, 2), dim3((unsigned)threads), 0,
                     static_cast<hipStream_t>(stream), a);
  return launched("keep");
}
