// tree_attention.hip -- attention of each sequence's newest tokens (a tree of
// drafted tokens; one token, a chain) over its quantised, paged K/V cache.
//
// The query rows of one sequence and kv head (new tokens x query heads of the
// group) share the keys they read, so they are the columns of the matrix-core
// products  S^T = K Q^T  and  O^T = V^T P^T  (v_mfma_f32_16x16x32_f16): a
// wavefront holds 16 RT rows of Q and of O in registers for its whole life and
// takes the keys 32 at a time.  In S^T a lane owns one row and 4 + 4 keys; those
// eight probabilities are, in the same lane and order, its part of the second
// product's operand, so P never leaves the registers.  The contraction may run
// over channels and keys in any order that both operands follow: a lane takes K in 16-byte
// pieces of a key's channels, V in pieces of 8 channels of each of its
// eight keys, which v_perm transposes while it widens the codes.  The lanes of an operand are
// neighbours in key, not in memory, so the blocks come through LDS: asked for a
// step ahead straight into it, moved to registers when they are there (loads of the
// operand's own layout cost an access for every lane: 64 sequences of up to 8192 tokens took 147 us with them).
//
// Exactness: int8 codes are fp16 values (the byte as a subnormal, one packed fma
// makes it code * 2^-9), their scales go to the fp32 scores (K) and to the
// probabilities (V); int4 codes times their 8-bit scales are fp16 values.  Q is
// scaled per row by a power of two into fp16's range.  So the only rounding
// below fp32 is that of the probabilities to fp16: they are kept near 2^11 of
// fp16's range relative to the running maximum and the largest V scale that the row has seen.
//
// What a row does not see must not reach it, whatever lies in memory there (a drafted token that was never stored, page 0
// in place of a bad one): its score becomes -inf and its probability 0, and the scale of a key that no row of the
// wavefront sees becomes 0 before it meets that 0, since 0 times an infinity or NaN is NaN.  Only blocks
// that reach past the older tokens, or have a tile without a page, pay for it.
//
// The running maximum moves only when a score passes it by 2^4 (one vote of the
// wavefront a step), so that the output is rarely rescaled.
//
// The keys of a sequence are cut into chunks, a workgroup each, whose four
// wavefronts (one where there are many cells of few keys) take every fourth block of 32 keys; the partial outputs of a few
// chunks are joined by the workgroup that finishes last, those of many by a second,
// small launch, in either case in chunk order.
//
// Bound for single tokens by memory: 64 sequences of up to 8192 int8 tokens (64 query heads over 8) 126 us, 5.4 TB/s, where
// the loads alone take 125 (they come as 8 KB a wavefront and step; twice that in flight gained nothing).  By the vector
// instructions that widen int4: 131001 tokens 35 us, 4.4 TB/s.  By the latency of its chain (lengths, pages, keys,
// join) for a short sequence: 511 tokens of 32 heads 7.4 us.  By the softmax's vector instructions and the operands' way out
// of LDS for many rows (see the wide kernel).
#include "serving.h"
#include "unpack.h"

namespace cl {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 32;         // keys of a wavefront's step
constexpr int kWaves = 4;
constexpr int kWideRows = 128;     // query rows of a workgroup of the wide kernel
constexpr float kNone = -3.4e38f;  // running maximum before any key
constexpr float kSlack = 4.f;      // log2 by which a score may pass the running maximum
constexpr int kProbBits = 11;      // probabilities are scaled by 2^11: with the slack at most 2^15

// Keys of a workgroup, so that one long sequence among short ones does not run alone at the end (64 sequences of up to 16000
// tokens, 64 heads over 8: 208 us; 214 with 2048, where the joins cost more, 215 with 8192).
constexpr int kMaxChunk = 4096;
// Chunks that the last workgroup of a cell joins; more are joined by a launch of their own, which spreads them over the card
// (one row of 32 heads, 511 keys in four chunks: 7.7 us, 9.7 with a launch; 64 rows of 8 x 8 heads, 2000 keys in eight: 23.8 and,
// with a launch, 22.5).
constexpr int kInline = 4;
constexpr int kFewKeys = 256;      // up to which many cells are a wavefront each
constexpr int kMaxCells = 65536;   // cells (sequence, kv head, row group) that may be joined so: their counters open the workspace
constexpr int kMaxSplits = 1024;   // chunks that a sequence's keys are cut into
// Bytes of partial outputs: past them the cells alone fill the card many times over, and longer chunks cost nothing (64 x 64 tokens of
// 64 heads over 8, one sequence of 131072 among short ones: 1.32 ms, 1.49 with the 4.3 GB that chunks of kMaxChunk want, 1.39
// with 1 GiB; 64 x 16 tokens 425 us, 434 with 1.1 GB, 475 with 256 MiB; 256 single tokens 514, 501 with 537 MB).
constexpr int64_t kMaxParts = (int64_t)512 << 20;

constexpr size_t kCounterBytes = kMaxCells * sizeof(uint32_t);
static_assert(kCounterBytes == CL_ATTENTION_COUNTER_BYTES, "the header's figure");

struct AttnArgs {
  const uint16_t* q;
  uint16_t* o;
  cl_kv_cache c;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  const int32_t* cu_q;
  const uint64_t* mask;
  uint32_t* counters;  // NULL: the join is a launch of its own
  float2* part_ml;
  float* part_o;
  int64_t q_token, q_head;
  int tokens, group, table_width, max_q, mask_words, bf16;
  int chunk, row_groups, rows_per_group, page_shift;
  float scale;
};

__device__ __forceinline__ f4 mfma16(const uint32_t (&a)[4], const uint32_t (&b)[4], f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, u4{a[0], a[1], a[2], a[3]}),
                                                __builtin_bit_cast(h8, u4{b[0], b[1], b[2], b[3]}), c, 0, 0, 0);
}

// Two outputs in one word.
__device__ __forceinline__ uint32_t pack16(int bf16, float x, float y) {
  return bf16 ? Elem<CL_BF16>::down(x) | (uint32_t)Elem<CL_BF16>::down(y) << 16
              : Elem<CL_F16>::down(x) | (uint32_t)Elem<CL_F16>::down(y) << 16;
}

// A sequence's rows and keys, and how its keys are cut: `splits` chunks of at least a.chunk keys, at most
// `max_splits` (a sequence longer than the launch was sized for gets longer chunks).
struct Range {
  int first, n_new, ctx, splits;
  uint32_t n, chunk;
};
__device__ __forceinline__ Range range_of(const AttnArgs& a, int first, int end, int ctx, int max_splits) {
  Range x;
  x.first = first;
  const int64_t n_new = (int64_t)end - x.first;
  x.n_new = x.first < 0 || n_new < 0 || n_new > a.max_q || x.first + n_new > a.tokens ? 0 : (int)n_new;
  x.ctx = max(ctx, 0);
  x.n = (uint32_t)x.ctx + x.n_new;
  x.chunk = a.chunk;
  if (x.n > x.chunk * (uint64_t)max_splits) {
    const uint32_t least = (x.n - 1) / max_splits + 1;
    x.chunk = (least + kBlock * kWaves - 1) / (kBlock * kWaves) * (kBlock * kWaves);
  }
  x.splits = x.n ? (int)((x.n - 1) / x.chunk + 1) : 0;
  return x;
}

// Largest of three, NaN if one is.  (fmaxf would first quiet each operand whose origin the compiler cannot see, an
// instruction apiece.)
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// Largest value of the four lanes that hold parts of one row (16 apart).
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Bits that any of 16 lanes side by side (a tile's rows) has.
__device__ __forceinline__ uint32_t any_of_rows(uint32_t v) {
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);   // quad_perm [1, 0, 3, 2]
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);   // quad_perm [2, 3, 0, 1]
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false);  // mirrored in 8
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false);  // mirrored in 16
  return v;
}

// Two bytes code + 128, as fp16 subnormals in the halves of a word -> code * 2^-9, exactly.
__device__ __forceinline__ uint32_t widen8(uint32_t pair) {
  const h2 a = __builtin_bit_cast(h2, pair);
  const h2 r = __builtin_elementwise_fma(a, h2{(_Float16)32768.f, (_Float16)32768.f}, h2{(_Float16)-0.25f, (_Float16)-0.25f});
  return __builtin_bit_cast(uint32_t, r);
}

// Nibbles `i` of the two halves of a word -> (nibble - 8) * s, exactly (s of 8 significant bits).  word8 is word >> 8: a nibble
// in the second place becomes 1024 + 16 nibble, which a fused multiply-add takes down as exactly as an addition
// 1024 + nibble.
__device__ __forceinline__ uint32_t widen4(uint32_t word, uint32_t word8, int i, h2 s) {
  const uint32_t w = i & 2 ? word8 : word;
  uint32_t exponent = 0x64006400u;
  asm("" : "+v"(exponent));  // in a register, so that mask and exponent are one instruction
  h2 c;
  if (i & 1)
    c = __builtin_elementwise_fma(__builtin_bit_cast(h2, (w & 0x00F000F0u) | exponent),
                                  h2{(_Float16)0.0625f, (_Float16)0.0625f}, h2{(_Float16)-72.f, (_Float16)-72.f});
  else
    c = __builtin_bit_cast(h2, (w & 0x000F000Fu) | exponent) - h2{(_Float16)1032.f, (_Float16)1032.f};
  return __builtin_bit_cast(uint32_t, c * s);
}

// Two fp16 values, an infinity or NaN replaced by fp16's largest.
__device__ __forceinline__ uint32_t finite(uint32_t pair) {
  const h2 most = {(_Float16)65504.f, (_Float16)65504.f};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_elementwise_min(__builtin_bit_cast(h2, pair), most), -most));
}

// The scales of a block of 32 keys, two tiles of 16, that a lane needs.
template <int KIND>
struct Scales;
template <>
struct Scales<CL_KV_INT8> {
  u2 k[2], v[2];  // fp16, of keys 4 (l / 16) .. of either tile
};
template <>
struct Scales<CL_KV_INT4> {
  uint32_t k[2];  // of key l % 16, the lane's channels
  uint32_t v[8];  // of keys 4 (l / 16) .. of either tile, the lane's channels
};

// What a lane keeps of RT query rows: row l % 16 of each tile.
template <int RT>
struct Rows {
  float rowc[RT];         // what turns a product of operands into a score, in log2
  float top[RT];          // running maximum of the scores
  float m[RT];            // it less log2(2^kProbBits / vref): sum and the outputs carry that factor, which the quotient loses
  float sum[RT];
  int tok[RT];            // its new token
  float vref[RT];         // a power of two above every V scale that the row has seen (int8; int4's V carries its scales)
};

// The first RT x 16 rows from `row0` of Q, raw.
template <int RT, int STEPS, typename Channel>
__device__ __forceinline__ void load_q(const AttnArgs& a, int first, int n_new, int hk, int row0, Channel channel, Rows<RT>& rows,
                                       u4 (&raw)[RT][STEPS]) {
  const int c16 = threadIdx.x & 15, G = a.group;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = row0 + 16 * r + c16;
    rows.tok[r] = row / G;
    const bool there = rows.tok[r] < n_new;  // otherwise the values are not used
    const uint16_t* qp = a.q + (int64_t)(first + (there ? rows.tok[r] : 0)) * a.q_token + (int64_t)(hk * G + row % G) * a.q_head;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) raw[r][s] = *reinterpret_cast<const u4*>(qp + channel(s));
  }
}

// Q as the second operand: scaled by a power of two into fp16's range.  An int4 piece of 8 channels is taken in the order
// 0, 4, 1, 5, 2, 6, 3, 7, as its nibbles come.
template <int KIND, int RT, int STEPS>
__device__ __forceinline__ void convert_q(const AttnArgs& a, const u4 (&raw)[RT][STEPS], Rows<RT>& rows, uint32_t (&q)[RT][STEPS][4]) {
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float f[STEPS][8], top = 0.f;
    bool fine = true;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint16_t e = (uint16_t)(raw[r][s][j / 2] >> (16 * (j % 2)));
        f[s][j] = a.bf16 ? Elem<CL_BF16>::up(e) : Elem<CL_F16>::up(e);
        fine = fine && fabsf(f[s][j]) < INFINITY;
        top = fmaxf(top, fabsf(f[s][j]));
      }
    }
    top = row_max(top);
    fine = row_max(fine ? 0.f : 1.f) == 0.f;
    int e = 0;
    (void)frexpf(top, &e);
    if (!(top > 0.f) || !fine) e = 0;
    // a row with an infinity or NaN is NaN; a negative scale turns Q around, so that rowc >= 0
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int lo = KIND == CL_KV_INT8 ? 2 * j : j, hi = KIND == CL_KV_INT8 ? 2 * j + 1 : j + 4;
        float x = ldexpf(f[s][lo], 14 - e), y = ldexpf(f[s][hi], 14 - e);
        if (a.scale < 0.f) x = -x, y = -y;
        if (a.scale == 0.f) x = y = 0.f;
        if (!fine) x = y = __builtin_nanf("");
        q[r][s][j] = __builtin_bit_cast(uint32_t, h2{(_Float16)x, (_Float16)y});
      }
    // above zero, so that a masked score of -inf stays what it is
    rows.rowc[r] = fmaxf(ldexpf(fabsf(a.scale) * 1.44269504f, e - 14 + (KIND == CL_KV_INT8 ? 9 : 0)), 1e-38f);
    rows.top[r] = rows.m[r] = kNone;
    rows.sum[r] = rows.vref[r] = 0.f;
  }
}

// Scores of a block of 32 keys from its products: K's scales (int8), and for a block that some rows do not see whole the
// masks.  s[r][t][i]: row l % 16 of tile r, key 16 t + 4 (l / 16) + i; j0: the block's first key; left: keys of it that exist;
// bad: tiles without a page.  ks, vs: the scales of those keys (int8); vtop: the largest vs that each row sees, of the lane's keys.
// Returns the block's keys that have a page and that some row of the wavefront sees; vs is 0 for the others.
template <int KIND, int RT>
__device__ __forceinline__ uint32_t finish_scores(const AttnArgs& a, const Range& range, const Rows<RT>& rows, const float (&ks)[8],
                                                  uint32_t j0, int left, int bad, bool special, f4 (&s)[RT][2], float (&vs)[8],
                                                  float (&vtop)[RT]) {
  const int g = (threadIdx.x & 63) >> 4;
  if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int r = 0; r < RT; ++r) s[r][j / 4][j % 4] *= ks[j];
  }
  if constexpr (KIND == CL_KV_INT8) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) top = max3(top, vs[j], vs[j + 1]);
#pragma unroll
    for (int r = 0; r < RT; ++r) vtop[r] = top;
  }
  if (!special) return ~0u;
  uint32_t seen[RT], any = 0;
  const int64_t rel = (int64_t)j0 - range.ctx;  // place of the block's first key among the new tokens
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    uint32_t see;  // keys of the block that the row sees
    if (!a.mask) {
      const int64_t cnt = rows.tok[r] - rel + 1;
      see = cnt >= 32 ? ~0u : cnt <= 0 ? 0u : (1u << cnt) - 1u;
    } else if (rel <= -32) {
      see = ~0u;
    } else {
      const uint64_t* w = a.mask + (int64_t)(range.first + min(rows.tok[r], range.n_new - 1)) * a.mask_words;
      if (rel < 0) {
        see = (uint32_t)(w[0] << -rel) | ((1u << -rel) - 1u);
      } else {
        const int at = (int)(rel >> 6), sh = (int)(rel & 63);
        uint64_t bits = at < a.mask_words ? w[at] >> sh : 0;
        if (sh > 32 && at + 1 < a.mask_words) bits |= w[at + 1] << (64 - sh);
        see = (uint32_t)bits;
      }
    }
    if (left < 32) see &= (1u << left) - 1u;
    if (rows.tok[r] >= range.n_new) see = 0;  // no such row
    seen[r] = see;
    any |= see;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int key = 16 * (j / 4) + 4 * g + j % 4;
      if (!((see >> key) & 1))
        s[r][j / 4][j % 4] = -INFINITY;
      else if ((bad >> (j / 4)) & 1)
        s[r][j / 4][j % 4] = __builtin_nanf("");
    }
  }
  any = any_of_rows(any) & ~((bad & 1 ? 0x0000FFFFu : 0u) | (bad & 2 ? 0xFFFF0000u : 0u));
  if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
    for (int r = 0; r < RT; ++r) vtop[r] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int key = 16 * (j / 4) + 4 * g + j % 4;
      if (!((any >> key) & 1)) vs[j] = 0.f;
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if ((seen[r] >> key) & 1) vtop[r] = fmaxf(vtop[r], vs[j]);
    }
  }
  return any;
}

// Probabilities of a block from its scores, as the operand of the second product; moves the running maximum, and with it
// sums and outputs, where a score passes it by more than the slack.
template <int KIND, int RT, int CB>
__device__ __forceinline__ void probabilities(const f4 (&s)[RT][2], const float (&vs)[8], const float (&vtop)[RT], Rows<RT>& rows,
                                              f4 (&o)[RT][CB], uint32_t (&p)[RT][4]) {
  float up[RT];
  bool move = false;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float t = max3(max3(s[r][0][0], s[r][0][1], s[r][0][2]), max3(s[r][0][3], s[r][1][0], s[r][1][1]),
                         max3(s[r][1][2], s[r][1][3], s[r][1][3]));
    up[r] = t * rows.rowc[r];
    move |= up[r] > rows.top[r] + kSlack;
    if constexpr (KIND == CL_KV_INT8) move |= vtop[r] > rows.vref[r];
  }
  if (__any(move)) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      // only a row that passed it, so that no row's roundings depend on another's
      float lift = -kProbBits;
      if constexpr (KIND == CL_KV_INT8) {
        const float v = row_max(vtop[r]);
        if (v > rows.vref[r]) rows.vref[r] = 2.f * __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0x7F800000u);
        lift = rows.vref[r] > 0.f ? __builtin_amdgcn_logf(rows.vref[r]) - kProbBits : 0.f;
      }
      const float high = row_max(up[r]);
      if (high > rows.top[r] + kSlack) rows.top[r] = high;
      const float next = rows.top[r] + lift, old = __builtin_amdgcn_exp2f(rows.m[r] - next);
      rows.m[r] = next;
      rows.sum[r] *= old;
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) o[r][cb] *= old;
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      e[j] = __builtin_amdgcn_exp2f(s[r][j / 4][j % 4] * rows.rowc[r] - rows.m[r]);
      rows.sum[r] += e[j];
      if constexpr (KIND == CL_KV_INT8) e[j] *= vs[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) p[r][j] = __builtin_bit_cast(uint32_t, h2{(_Float16)e[2 * j], (_Float16)e[2 * j + 1]});
  }
}

// 16 bytes of each lane straight into LDS, lane l's at `to` + 16 l; not kept in the caches (aux 2), which is worth a tenth of
// the rate on long contexts: 64 sequences of up to 8192 tokens 142 -> 127 us.
__device__ __forceinline__ void load_to_lds(const uint8_t* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void*)from, (__attribute__((address_space(3))) void*)to,
                                   16, 0, 2);
}

// Device-scope (all XCDs) accesses of two floats.
__device__ __forceinline__ void store_dev2(float2* p, float x, float y) {
  const uint64_t v = (uint64_t)__builtin_bit_cast(uint32_t, y) << 32 | __builtin_bit_cast(uint32_t, x);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_dev2(const float2* p) {
  const uint64_t v = __hip_atomic_load(const_cast<uint64_t*>(reinterpret_cast<const uint64_t*>(p)), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__builtin_bit_cast(float, (uint32_t)v), __builtin_bit_cast(float, (uint32_t)(v >> 32)));
}

// Waits for every load asked for so far, those into LDS among them.
__device__ __forceinline__ void wait_loads() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Waits for the reads of LDS, so that a load may overwrite what they read.
__device__ __forceinline__ void wait_lds() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

template <int KIND, int D, int RT, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 2) tree_attention_kernel(AttnArgs a) {
  constexpr int STEPS = D / 32;  // matrix-core steps of a score tile
  constexpr int CB = D / 16;     // channel blocks of the output; lane c of a block's 16 rows is channel CB c + block
  constexpr int ROWS = 16 * RT, STRIDE = D + 4;
  constexpr int ROWB = KIND == CL_KV_INT8 ? D : D / 2;  // bytes of a (token, head)
  constexpr int SC = KIND == CL_KV_INT8 ? 1 : D / 32;
  constexpr int PIECES = ROWB / 16, TILEB = 16 * ROWB;
  // a block of K and V of each wavefront, and later its output
  constexpr int BLOCKB = 4 * TILEB;
  constexpr size_t KVBYTES = (size_t)WAVES * BLOCKB, OBYTES = (size_t)WAVES * ROWS * STRIDE * 4;
  __shared__ __align__(1024) uint8_t s_mem[KVBYTES > OBYTES ? KVBYTES : OBYTES];
  float (*const s_o)[ROWS][STRIDE] = reinterpret_cast<float (*)[ROWS][STRIDE]>(s_mem);
  __shared__ float2 s_ml[WAVES][ROWS];
  __shared__ int s_last;

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, c16 = l & 15, g = l >> 4;
  const int b = blockIdx.y, hk = blockIdx.x % a.c.heads, rg = blockIdx.x / a.c.heads;
  const int split = blockIdx.z;

  // pages of the wavefront's next 64 tiles of 16 keys, one to a lane: -1 outside the cache or the table
  int pages = 0;
  const auto load_pages = [&](uint32_t from, int i) {
    const uint32_t at = from + (uint32_t)(wave + WAVES * (i + (l >> 1))) * kBlock + 16 * (l & 1);
    const uint32_t col = at >> a.page_shift;
    int p = col < (uint32_t)a.table_width ? a.block_table[(int64_t)b * a.table_width + col] : -1;
    pages = p < a.c.pages ? p : -1;
  };
  // the first of them are asked for together with the lengths, which they do not wait for
  load_pages((uint32_t)split * a.chunk, 0);
  const Range range = range_of(a, a.cu_q[b], a.cu_q[b + 1], a.ctx_lens[b], gridDim.z);
  const int first = range.first, n_new = range.n_new, ctx = range.ctx, splits = range.splits;
  const uint32_t n = range.n, chunk = range.chunk;
  const int G = a.group, rows = min(n_new * G - rg * ROWS, ROWS);  // rows of this workgroup that exist
  if (rows <= 0 || split >= splits) return;
  const uint32_t k0 = split * chunk;  // 32-bit places: a sequence has fewer than 2^31 + 256 tokens
  const int blocks = (int)((min(n - k0, chunk) + kBlock - 1) / kBlock);
  if (chunk != (uint32_t)a.chunk) load_pages(k0, 0);

  const uint8_t* const kb = static_cast<const uint8_t*>(a.c.k);
  const uint8_t* const vb = static_cast<const uint8_t*>(a.c.v);
  const int tiles_shift = a.page_shift - 4;  // tiles in a page
  // The path through LDS: lane l of a load fills bytes 16 l .. of its kilobyte and picks its global address to suit.
  // A 16-byte piece j of row r of a K tile lies at place j ^ swizzle(r) of its row, which spreads the 16 rows that 16
  // lanes read together over all banks; row r of a V tile lies at row turn(r), which does so for the rows
  // 0, 4, 8, 12 that four lane groups read together (turn is its own inverse).
  const auto swizzle = [](uint32_t r) -> uint32_t { return (r * ROWB / 256) & (PIECES - 1); };
  const auto turn = [](uint32_t r) -> uint32_t { return r ^ ((r >> 2) & 3); };
  uint8_t* const buf = s_mem + wave * BLOCKB;
  constexpr int LOADS = TILEB >= 1024 ? TILEB / 1024 : 1;  // of a tile; where a tile is half a load (dim 64 int4), of two
  uint32_t kfrom[LOADS], vfrom[LOADS];
#pragma unroll
  for (int q = 0; q < LOADS; ++q) {
    const uint32_t r = (q * 64 + l) / PIECES % 16, j = l % PIECES;
    kfrom[q] = r * ROWB + ((j ^ swizzle(r)) << 4);
    vfrom[q] = turn(r) * ROWB + (j << 4);
  }
  // where the lane reads: of K, key l % 16, its first piece (its second one, for 128-byte rows, is 4 pieces on); of V, key
  // 4 (l / 16) + j, a sixteenth of the row
  const uint32_t kread = c16 * ROWB + (((KIND == CL_KV_INT4 && D == 64 ? g / 2 : g) ^ swizzle(c16)) << 4) +
                         (KIND == CL_KV_INT4 && D == 64 ? 8 * (g % 2) : 0);
  uint32_t vread[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) vread[j] = turn(4 * g + j) * ROWB + ROWB / 16 * c16;

  // Row of the cache where tile t of step i starts.  A tile past the sequence's end, or without a page, is read
  // from page 0, which is there; its keys are masked, or the rows that see them become NaN.
  const auto row_of = [&](int i, int t, int* bad) -> int64_t {
    const int blk = wave + WAVES * i;
    const uint32_t at = k0 + (uint32_t)blk * kBlock + 16 * t;
    int page = __builtin_amdgcn_readlane(pages, 2 * (i & 31) + t);
    if (blk >= blocks || at >= n) {
      page = 0;
    } else if (page < 0) {
      page = 0;
      *bad |= 1 << t;
    }
    const int tile = (int)(at >> 4) & ((1 << tiles_shift) - 1);
    return (((int64_t)page * a.c.heads + hk) << a.page_shift) + (tile << 4);
  };
  // Asks for step i's block: K and V into LDS, the scales into registers.  Returns the tiles (bits) without a page.
  const auto load = [&](int i, Scales<KIND>& x) -> int {
    if (i > 0 && (i & 31) == 0) load_pages(k0, i);
    int bad = 0;
    int64_t row[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) row[t] = row_of(i, t, &bad);
    uint8_t* const to = buf;
    if constexpr (TILEB >= 1024) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int q = 0; q < LOADS; ++q) {
          load_to_lds(kb + row[t] * ROWB + kfrom[q], to + t * TILEB + 1024 * q);
          load_to_lds(vb + row[t] * ROWB + vfrom[q], to + (2 + t) * TILEB + 1024 * q);
        }
    } else {
      const int64_t mine = l < 32 ? row[0] : row[1];
      load_to_lds(kb + mine * ROWB + kfrom[0], to);
      load_to_lds(vb + mine * ROWB + vfrom[0], to + 2 * TILEB);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint16_t* ksp = a.c.k_scale + row[t] * SC;
      const uint16_t* vsp = a.c.v_scale + row[t] * SC;
      if constexpr (KIND == CL_KV_INT8) {
        x.k[t] = *reinterpret_cast<const u2*>(ksp + 4 * g);
        x.v[t] = *reinterpret_cast<const u2*>(vsp + 4 * g);
      } else {
        x.k[t] = ksp[(uint32_t)(c16 * SC + (D == 128 ? g : g / 2))];
#pragma unroll
        for (int j = 0; j < 4; ++j) x.v[4 * t + j] = vsp[(uint32_t)((4 * g + j) * SC + CB * c16 / 32)];
      }
    }
    return bad;
  };

  // ---- the first block and raw Q
  const int steps = wave < blocks ? (blocks - wave + WAVES - 1) / WAVES : 0;
  Scales<KIND> sc_next;
  int bad_next = 0;
  if (steps > 0) bad_next = load(0, sc_next);
  Rows<RT> st;
  u4 raw[RT][STEPS];
  load_q(a, first, n_new, hk, rg * ROWS,
         [&](int s) { return KIND == CL_KV_INT8 ? (s / 2) * 64 + 16 * g + (s % 2) * 8 : (D / 4) * g + 8 * s; }, st, raw);
  uint32_t q[RT][STEPS][4];
  convert_q<KIND>(a, raw, st, q);
  f4 o[RT][CB];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) o[r][cb] = f4{0.f, 0.f, 0.f, 0.f};

  for (int i = 0; i < steps; ++i) {
    // the block moves from LDS into registers, then the next one flies for a whole step
    wait_loads();
    u4 kr[2][KIND == CL_KV_INT8 ? D / 64 : 1];
    u2 vr[8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* const kt = buf + t * TILEB;
      if constexpr (KIND == CL_KV_INT4 && D == 64) {
        const u2 half = *reinterpret_cast<const u2*>(kt + kread);
        kr[t][0].x = half.x, kr[t][0].y = half.y;
      } else {
        kr[t][0] = *reinterpret_cast<const u4*>(kt + kread);
        if constexpr (KIND == CL_KV_INT8 && D == 128) kr[t][1] = *reinterpret_cast<const u4*>(kt + (kread ^ 64));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t* const at = buf + (2 + j / 4) * TILEB + vread[j % 4];
      if constexpr (KIND == CL_KV_INT8 && D == 128)
        vr[j] = *reinterpret_cast<const u2*>(at);
      else if constexpr (KIND == CL_KV_INT4 && D == 64)
        vr[j].x = *reinterpret_cast<const uint16_t*>(at);
      else
        vr[j].x = *reinterpret_cast<const uint32_t*>(at);
    }
    wait_lds();
    const Scales<KIND> sc = sc_next;
    const int bad = bad_next;
    if (i + 1 < steps) bad_next = load(i + 1, sc_next);
    const uint32_t j0 = k0 + (uint32_t)(wave + WAVES * i) * kBlock;
    const int left = (int)min(n - j0, (uint32_t)kBlock);         // keys of the block that exist
    const bool special = j0 + kBlock > (uint32_t)ctx || bad;     // some rows may not see some keys

    // ---- scores
    f4 s[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r) s[r][0] = s[r][1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        uint32_t k[4];
        if constexpr (KIND == CL_KV_INT8) {
          const u4 raw = kr[t][st / 2];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            k[j] = widen8(perm(0, raw[2 * (st % 2) + j / 2], j % 2 ? 0x0C030C02u : 0x0C010C00u));
        } else {
          const h2 ks = __builtin_bit_cast(h2, sc.k[t] | sc.k[t] << 16);
          const uint32_t w = kr[t][0][st], w8 = w >> 8;
#pragma unroll
          for (int j = 0; j < 4; ++j) k[j] = widen4(w, w8, j, ks);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r][t] = mfma16(k, q[r][st], s[r][t]);
      }
    }
    float ks[8], vs[8], vtop[RT];
    uint32_t p[RT][4];
    if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ks[j] = Elem<CL_F16>::up((uint16_t)(sc.k[j / 4][j % 4 / 2] >> (16 * (j % 2))));
        vs[j] = Elem<CL_F16>::up((uint16_t)(sc.v[j / 4][j % 4 / 2] >> (16 * (j % 2))));
      }
    }
    const uint32_t seen = finish_scores<KIND>(a, range, st, ks, j0, left, bad, special, s, vs, vtop);
    probabilities<KIND>(s, vs, vtop, st, o, p);
    // ---- output
    if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        uint32_t v[4];
        const uint32_t sel = 0x0C040C00u + 0x00010001u * (cb % 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = widen8(perm(vr[2 * j + 1][cb / 4], vr[2 * j][cb / 4], sel));
#pragma unroll
        for (int r = 0; r < RT; ++r) o[r][cb] = mfma16(v, p[r], o[r][cb]);
      }
    } else {
      h2 mul[4];
      uint32_t vsc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) vsc[j] = sc.v[j];
      if (special) {  // where no row sees a token the scale may be anything
        asm volatile("");  // a branch, not eight selects a block
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!((seen >> (16 * (j / 4) + 4 * g + j % 4)) & 1)) vsc[j] = 0;
      }
      uint32_t lo[4], hi[4];  // channels 0..3 and 4..7 of two keys, one in each half
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mul[j] = __builtin_bit_cast(h2, vsc[2 * j] | vsc[2 * j + 1] << 16);
        lo[j] = perm(vr[2 * j + 1].x, vr[2 * j].x, 0x05040100u);
        hi[j] = perm(vr[2 * j + 1].x, vr[2 * j].x, 0x07060302u);
      }
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = cb < 4 ? lo[j] : hi[j];
          v[j] = widen4(w, w >> 8, cb % 4, mul[j]);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) o[r][cb] = mfma16(v, p[r], o[r][cb]);
      }
    }
  }

  // ---- join the four wavefronts
  __syncthreads();  // the blocks' memory becomes the outputs'
  constexpr float unit = KIND == CL_KV_INT8 ? 512.f : 1.f;  // codes entered as code * 2^-9
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float l_row = row_sum(st.sum[r]);
    const int row = 16 * r + c16;
    if (g == 0) s_ml[wave][row] = make_float2(st.m[r], l_row);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int c4 = 0; c4 < CB; c4 += 4)
        *reinterpret_cast<f4*>(&s_o[wave][row][CB * (4 * g + i) + c4]) =
            f4{o[r][c4][i], o[r][c4 + 1][i], o[r][c4 + 2][i], o[r][c4 + 3][i]} * unit;
    }
  }
  __syncthreads();
  constexpr int PARTS = D / 8;  // threads of a row, 8 channels each
  const int64_t cell = ((int64_t)b * a.c.heads + hk) * a.row_groups + rg;
  const int ch = 8 * (tid % PARTS);
  const auto store = [&](int row, const float (&x)[8], float inv) {
    const int at = rg * ROWS + row;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack16(a.bf16, x[2 * j] * inv, x[2 * j + 1] * inv);
    uint16_t* op = a.o + ((int64_t)(first + at / G) * (a.c.heads * G) + hk * G + at % G) * D + ch;
    *reinterpret_cast<u4*>(op) = u4{w[0], w[1], w[2], w[3]};
  };
  for (int row = tid / PARTS; row < rows; row += 64 * WAVES / PARTS) {
    float top = kNone, w[WAVES], den = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < WAVES; ++v) top = fmaxf(top, s_ml[v][row].x);
#pragma unroll
    for (int v = 0; v < WAVES; ++v) {
      w[v] = __builtin_amdgcn_exp2f(s_ml[v][row].x - top);
      den += w[v] * s_ml[v][row].y;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] += w[v] * s_o[v][row][ch + j];
    }
    if (splits == 1) {
      store(row, x, den == 0.f ? 0.f : 1.f / den);
    } else {
      const int64_t at = (cell * gridDim.z + split) * ROWS + row;
      float* const op = a.part_o + at * D + ch;
      if (a.counters) {  // read by a workgroup of this launch
        if (ch == 0) store_dev2(a.part_ml + at, top, den);
#pragma unroll
        for (int j = 0; j < 8; j += 2) store_dev2(reinterpret_cast<float2*>(op + j), x[j], x[j + 1]);
      } else {
        if (ch == 0) a.part_ml[at] = make_float2(top, den);
        *reinterpret_cast<f4*>(op) = f4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f4*>(op + 4) = f4{x[4], x[5], x[6], x[7]};
      }
    }
  }
  if (splits == 1 || !a.counters) return;
  // ---- few chunks: the workgroup that comes last joins them
  wait_stores();
  __syncthreads();
  if (tid == 0) {
    const uint32_t before = __hip_atomic_fetch_add(&a.counters[cell], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_last = before == (uint32_t)splits - 1;
    if (s_last) __hip_atomic_store(&a.counters[cell], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!s_last) return;
  for (int row = tid / PARTS; row < rows; row += 64 * WAVES / PARTS) {
    float mv[kInline], lv[kInline], x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, top = kNone, den = 0.f;
    float2 part[kInline][4];
#pragma unroll
    for (int v = 0; v < kInline; ++v) {
      const int64_t at = (cell * gridDim.z + min(v, splits - 1)) * ROWS + row;
      const float2 ml = load_dev2(a.part_ml + at);
      mv[v] = v < splits ? ml.x : kNone;
      lv[v] = v < splits ? ml.y : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) part[v][j] = load_dev2(reinterpret_cast<const float2*>(a.part_o + at * D + ch + 2 * j));
    }
#pragma unroll
    for (int v = 0; v < kInline; ++v) top = fmaxf(top, mv[v]);
#pragma unroll
    for (int v = 0; v < kInline; ++v) {
      const float w = v < splits ? __builtin_amdgcn_exp2f(mv[v] - top) : 0.f;
      den += w * lv[v];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (v < splits) x[2 * j] += w * part[v][j].x, x[2 * j + 1] += w * part[v][j].y;
      }
    }
    store(row, x, den == 0.f ? 0.f : 1.f / den);
  }
}

// Many query rows of a kv head and one sequence (a tree of a grouped model): a workgroup has 128 rows, 32 to a wavefront, and all of them read the
// same keys.  Its threads widen a block of 32 keys together, K as rows of fp16 and V transposed, into one of two LDS
// buffers while the products run on the other; so a code is widened once for 128 rows, and an operand is one 16-byte read.
// A tree of 64 over 61441 int8 tokens, 64 query heads over 8: 184 us and 10 of the join, 0.66 PFLOP/s.  Bound by what two wavefronts to a SIMD do
// not overlap: per block of 32 keys 1.4 us for the eight of a CU, where the products alone take 0.76, with their
// operands from LDS 0.97, with the softmax instead 0.98 (one wavefront to a SIMD with 64 rows, half the LDS reads for a
// product, spills: 293 us; K's products a block ahead of the softmax 201; three to a SIMD spill).
template <int KIND, int D>
__global__ void __launch_bounds__(256, 2) tree_attention_wide_kernel(AttnArgs a) {
  constexpr int RT = 2, STEPS = D / 32, CB = D / 16, ROWS = kWideRows;
  constexpr int ROWB = KIND == CL_KV_INT8 ? D : D / 2, SC = KIND == CL_KV_INT8 ? 1 : D / 32;
  constexpr int KB = 32 * D * 2;        // bytes of a block's K as fp16
  constexpr int VS = 80;                // bytes between the channels of a block's V: 32 keys and padding
  constexpr int KT = ROWB / 8;          // bytes of K that a thread widens: an eighth of a row
  constexpr int VC = D / 32;            // channels of V that a thread widens, of four keys
  __shared__ __align__(1024) uint8_t s_mem[2][KB + D * VS];
  __shared__ __align__(16) float s_scale[2][2][32];  // int8: K's and V's scales of a block
  __shared__ int s_bad[2];                           // its tiles without a page

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, c16 = l & 15, g = l >> 4;
  const int b = blockIdx.y, hk = blockIdx.x % a.c.heads, rg = blockIdx.x / a.c.heads, split = blockIdx.z;
  const Range range = range_of(a, a.cu_q[b], a.cu_q[b + 1], a.ctx_lens[b], gridDim.z);
  const int first = range.first, n_new = range.n_new;
  const int G = a.group, rows_left = n_new * G - rg * ROWS;
  if (rows_left <= 0 || split >= range.splits) return;
  const uint32_t n = range.n, k0 = split * range.chunk;
  const int blocks = (int)((min(n - k0, range.chunk) + kBlock - 1) / kBlock);
  const bool active = wave * 32 < rows_left;  // whether the wavefront has rows

  // pages of the next 64 tiles of 16 keys, one to a lane: -1 outside the cache or the table, 0 past the end
  int pages = 0;
  const auto load_pages = [&](int i) {
    const uint32_t at = k0 + (uint32_t)(i + (l >> 1)) * kBlock + 16 * (l & 1), col = at >> a.page_shift;
    int p = 0;
    if (i + (l >> 1) < blocks && at < n) {
      p = col < (uint32_t)a.table_width ? a.block_table[(int64_t)b * a.table_width + col] : -1;
      if (p < 0 || p >= a.c.pages) p = -1;
    }
    pages = p;
  };
  const int in_page = (1 << (a.page_shift - 4)) - 1;
  const auto row_of = [&](int i, int t, int* bad) -> int64_t {
    int page = __builtin_amdgcn_readlane(pages, 2 * (i & 31) + t);
    if (page < 0) *bad |= 1 << t, page = 0;
    const int tile = (int)((k0 + (uint32_t)i * kBlock) >> 4) + t;
    return (((int64_t)page * a.c.heads + hk) << a.page_shift) + ((tile & in_page) << 4);
  };

  // ---- a thread's share of a block: an eighth of K's row tid / 8; VC channels of V's keys 4 (tid / 32) ..  A wavefront's share
  // lies in one tile
  const int krow = tid >> 3, kpart = tid & 7, vkey = 4 * (tid >> 5), vch = VC * (tid & 31);
  struct Raw {
    u4 k;
    uint32_t v[4];
    uint16_t ks, vs[4];  // int4; int8: ks is K's or V's scale of key tid % 32, by the first 64 threads
    int bad;
  };
  const auto load = [&](int i, Raw& x) {
    if ((i & 31) == 0) load_pages(i);
    x.bad = 0;
    int64_t row[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) row[t] = row_of(i, t, &x.bad);
    const int64_t mine = wave < 2 ? row[0] : row[1];
    const uint8_t* kp = static_cast<const uint8_t*>(a.c.k) + mine * ROWB + (uint32_t)((krow & 15) * ROWB + kpart * KT);
    if constexpr (KT == 16) {
      x.k = *reinterpret_cast<const u4*>(kp);
    } else if constexpr (KT == 8) {
      const u2 w = *reinterpret_cast<const u2*>(kp);
      x.k.x = w.x, x.k.y = w.y;
    } else {
      x.k.x = *reinterpret_cast<const uint32_t*>(kp);
    }
    const uint8_t* vp = static_cast<const uint8_t*>(a.c.v) + mine * ROWB +
                        (uint32_t)((vkey & 15) * ROWB + (KIND == CL_KV_INT8 ? vch : vch / 2));
    constexpr int VB = KIND == CL_KV_INT8 ? VC : VC / 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (VB == 4)
        x.v[j] = *reinterpret_cast<const uint32_t*>(vp + j * ROWB);
      else if constexpr (VB == 2)
        x.v[j] = *reinterpret_cast<const uint16_t*>(vp + j * ROWB);
      else
        x.v[j] = vp[j * ROWB];
    }
    if constexpr (KIND == CL_KV_INT8) {
      if (wave == 0) x.ks = (l < 32 ? a.c.k_scale : a.c.v_scale)[((l & 16) ? row[1] : row[0]) + (l & 15)];
    } else {
      x.ks = a.c.k_scale[mine * SC + (krow & 15) * SC + kpart * (D / 8) / 32];
#pragma unroll
      for (int j = 0; j < 4; ++j) x.vs[j] = a.c.v_scale[mine * SC + ((vkey & 15) + j) * SC + vch / 32];
    }
  };
  // Widens it into a buffer.  K: row r's 16-byte piece j (8 channels) at place j ^ (r mod pieces); V: channel c's 32 keys in the
  // order of the second product's slots (slot 8 g + i is key 4 g + i, slot 8 g + 4 + i key 16 + 4 g + i).  The padding
  // spreads the channels that lanes read together over the banks, and the turn (lanes start at different ones of
  // their channels) those that they write together.
  constexpr int PIECES = D / 8;
  const auto widen = [&](const Raw& x, int i) {
    uint8_t* const to = s_mem[i & 1];
    if (tid == 0) s_bad[i & 1] = x.bad;
    if (KIND == CL_KV_INT8 && wave == 0) (&s_scale[i & 1][0][0])[l] = Elem<CL_F16>::up(x.ks);
    u4 piece[D / 64];
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (KIND == CL_KV_INT8)
          piece[p][j] = widen8(perm(0, x.k[2 * p + j / 2], j % 2 ? 0x0C030C02u : 0x0C010C00u));
        else
          piece[p][j] = widen4(x.k[p], x.k[p] >> 8, j, __builtin_bit_cast(h2, (uint32_t)x.ks * 0x10001u));
      }
      const uint32_t j = kpart * (D / 64) + p;
      *reinterpret_cast<u4*>(to + krow * (2 * D) + ((j ^ (krow & (PIECES - 1))) << 4)) = piece[p];
    }
    uint8_t* const vt = to + KB + (16 * ((vkey & 15) >> 2) + 8 * (vkey >> 4));
    const int turn = VC == 4 ? (tid & 31) >> 2 : (tid & 31) >> 3;
    if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        const int own = (c + turn) & (VC - 1);
        const uint32_t sel = 0x0C040C00u + 0x00010001u * own;
        *reinterpret_cast<u2*>(vt + (vch + own) * VS) = u2{widen8(perm(x.v[1], x.v[0], sel)), widen8(perm(x.v[3], x.v[2], sel))};
      }
    } else {
      h2 mul[2];
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mul[j] = __builtin_bit_cast(h2, (uint32_t)x.vs[2 * j] | (uint32_t)x.vs[2 * j + 1] << 16);
        w[j] = x.v[2 * j] | x.v[2 * j + 1] << 16;
      }
      u2 val[VC];
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        const int own = (c + turn) & (VC - 1);
        val[c] = u2{widen4(w[0] >> 4 * own, 0, 0, mul[0]), widen4(w[1] >> 4 * own, 0, 0, mul[1])};
      }
      // Which keys of the block no row sees is not known yet.  There anything may come out, so it is made finite (the
      // probabilities there are 0); a stored value is and stays as it is.
      if (k0 + (uint32_t)(i + 1) * kBlock > (uint32_t)range.ctx || x.bad) {
        asm volatile("");  // a branch
#pragma unroll
        for (int c = 0; c < VC; ++c) val[c] = u2{finite(val[c].x), finite(val[c].y)};
      }
#pragma unroll
      for (int c = 0; c < VC; ++c)
        *reinterpret_cast<u2*>(vt + (vch + ((c + turn) & (VC - 1))) * VS) = val[c];
    }
  };
  Raw x;
  load(0, x);
  Rows<RT> st;
  u4 raw[RT][STEPS];
  load_q(a, first, n_new, hk, rg * ROWS + 32 * wave, [&](int s) { return 32 * s + 8 * g; }, st, raw);
  uint32_t q[RT][STEPS][4];
  convert_q<KIND>(a, raw, st, q);
  f4 o[RT][CB];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) o[r][cb] = f4{0.f, 0.f, 0.f, 0.f};
  widen(x, 0);
  if (blocks > 1) load(1, x);

  for (int i = 0; i < blocks; ++i) {
    __syncthreads();  // block i is widened; the other buffer is free
    if (i + 1 < blocks) widen(x, i + 1);
    if (i + 2 < blocks) load(i + 2, x);
    if (!active) continue;
    const uint8_t* const kt = s_mem[i & 1];
    const uint8_t* const vt = kt + KB;
    const uint32_t j0 = k0 + (uint32_t)i * kBlock;
    const int left = (int)min(n - j0, (uint32_t)kBlock), bad = __builtin_amdgcn_readfirstlane(s_bad[i & 1]);
    const bool special = j0 + kBlock > (uint32_t)range.ctx || bad;
    f4 s[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r) s[r][0] = s[r][1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        const u4 w = *reinterpret_cast<const u4*>(kt + (16 * t + c16) * (2 * D) + (((4 * k + g) ^ (c16 & (PIECES - 1))) << 4));
        const uint32_t kk[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r][t] = mfma16(kk, q[r][k], s[r][t]);
      }
    float ks[8], vs[8], vtop[RT];
    if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const f4 k4 = *reinterpret_cast<const f4*>(&s_scale[i & 1][0][16 * t + 4 * g]);
        const f4 v4 = *reinterpret_cast<const f4*>(&s_scale[i & 1][1][16 * t + 4 * g]);
#pragma unroll
        for (int j = 0; j < 4; ++j) ks[4 * t + j] = k4[j], vs[4 * t + j] = v4[j];
      }
    }
    u4 vf[CB - 2];  // V's operands, asked for before the softmax as far as there are registers
#pragma unroll
    for (int cb = 0; cb < CB - 2; ++cb) vf[cb] = *reinterpret_cast<const u4*>(vt + (16 * cb + c16) * VS + 16 * g);
    uint32_t p[RT][4];
    finish_scores<KIND>(a, range, st, ks, j0, left, bad, special, s, vs, vtop);
    probabilities<KIND>(s, vs, vtop, st, o, p);
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      const u4 w = cb < CB - 2 ? vf[cb < CB - 2 ? cb : 0] : *reinterpret_cast<const u4*>(vt + (16 * cb + c16) * VS + 16 * g);
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int r = 0; r < RT; ++r) o[r][cb] = mfma16(v, p[r], o[r][cb]);
    }
  }
  if (!active) return;

  // ---- each wavefront has its rows whole: lane (row l % 16, channels 16 cb + 4 g ..)
  constexpr float unit = KIND == CL_KV_INT8 ? 512.f : 1.f;  // codes entered as code * 2^-9
  const int64_t cell = ((int64_t)b * a.c.heads + hk) * a.row_groups + rg;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = 32 * wave + 16 * r + c16;
    const float den = row_sum(st.sum[r]);
    if (row >= rows_left) continue;
    if (range.splits == 1) {
      const float inv = den == 0.f ? 0.f : unit / den;
      const int at = rg * ROWS + row;
      uint16_t* op = a.o + ((int64_t)(first + at / G) * (a.c.heads * G) + hk * G + at % G) * D + 4 * g;
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
        *reinterpret_cast<u2*>(op + 16 * cb) = u2{pack16(a.bf16, o[r][cb][0] * inv, o[r][cb][1] * inv),
                                                 pack16(a.bf16, o[r][cb][2] * inv, o[r][cb][3] * inv)};
    } else {
      const int64_t at = (cell * gridDim.z + split) * ROWS + row;
      if (g == 0) a.part_ml[at] = make_float2(st.m[r], den);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) *reinterpret_cast<f4*>(a.part_o + at * D + 16 * cb + 4 * g) = o[r][cb] * unit;
    }
  }
}

// Joins the partial outputs of a row's chunks, in chunk order within each of eight strands and the strands in
// order: 32 lanes (dim 128) or 16 hold four channels each.
template <int D>
__global__ void __launch_bounds__(256) tree_attention_join_kernel(AttnArgs a, int max_splits) {
  constexpr int LANES = D / 4, STRANDS = 256 / LANES;
  __shared__ float s_w[kMaxSplits];
  __shared__ __align__(16) f4 s_x[STRANDS][LANES];
  __shared__ float s_red[2 * kWaves];
  const int tid = threadIdx.x, cell = blockIdx.x, row = blockIdx.y;
  const int rg = cell % a.row_groups, hk = cell / a.row_groups % a.c.heads, b = cell / a.row_groups / a.c.heads;
  const Range x = range_of(a, a.cu_q[b], a.cu_q[b + 1], a.ctx_lens[b], max_splits);
  const int G = a.group, at = rg * a.rows_per_group + row;
  if (x.splits < 2 || at >= x.n_new * G) return;
  const int64_t base = (int64_t)cell * max_splits * a.rows_per_group + row;
  const int ch = tid % LANES, strand = tid / LANES;
  float top = kNone;
  for (int v = tid; v < x.splits; v += 256) top = fmaxf(top, a.part_ml[base + (int64_t)v * a.rows_per_group].x);
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  if (tid % 64 == 0) s_red[tid / 64] = top;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kWaves; ++v) top = fmaxf(top, s_red[v]);
  float den = 0.f;
  for (int v = tid; v < x.splits; v += 256) {
    const float2 ml = a.part_ml[base + (int64_t)v * a.rows_per_group];
    const float w = __builtin_amdgcn_exp2f(ml.x - top);
    s_w[v] = w;
    den += w * ml.y;
  }
  for (int d = 1; d < 64; d <<= 1) den += __shfl_xor(den, d);
  if (tid % 64 == 0) s_red[kWaves + tid / 64] = den;
  __syncthreads();
  den = 0.f;
#pragma unroll
  for (int v = 0; v < kWaves; ++v) den += s_red[kWaves + v];
  f4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int v = strand; v < x.splits; v += STRANDS) {
    const f4 part = *reinterpret_cast<const f4*>(a.part_o + (base + (int64_t)v * a.rows_per_group) * D + 4 * ch);
    sum += part * s_w[v];
  }
  s_x[strand][ch] = sum;
  __syncthreads();
  if (strand > 0) return;
#pragma unroll
  for (int v = 1; v < STRANDS; ++v) sum += s_x[v][ch];
  const float inv = den == 0.f ? 0.f : 1.f / den;
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) w[j] = pack16(a.bf16, sum[2 * j] * inv, sum[2 * j + 1] * inv);
  uint16_t* op = a.o + ((int64_t)(x.first + at / G) * (a.c.heads * G) + hk * G + at % G) * D + 4 * ch;
  *reinterpret_cast<u2*>(op) = u2{w[0], w[1]};
}

// How a launch is cut: rows to a workgroup, row groups, chunks of keys.
struct AttnPlan {
  bool wide;
  int group_rows, row_groups, splits, chunk;  // rows of a row group (a workgroup)
  int waves;                                  // wavefronts of one of 16 rows
  int64_t cells;
  bool joined_inline;
  size_t ml_bytes, o_bytes, need;
};

AttnPlan plan_attention(int64_t sequences, int q_heads, int heads, int dim, int max_q, int64_t max_ctx) {
  AttnPlan p;
  const int64_t rows = (int64_t)max_q * (q_heads / heads);
  const int64_t keys = max_ctx + max_q, unit = kBlock * kWaves, ones = (keys + unit - 1) / unit;
  // Rows to a workgroup: more of them read and widen a key once for more rows, but leave fewer workgroups with longer
  // chains to their end.  128 pay for one sequence, whose keys are cut evenly, where a CU has 7 steps or more of them (64
  // tokens of 8 x 8 heads: 16000 keys 67 us against 73 with 32 rows, 4000 keys 37 against 33), not for several, whose
  // lengths differ (8 such sequences of up to 8000 keys: 173 against 100; two of up to 30000: 189 against 201, of 8000 70 against
  // 65); 32 where a CU has more than 20 steps of 16 rows (16 tokens of 8 x 8 heads: 16000 keys 30.8 us
  // against 33.8 with 16 rows, 8000 keys 25.3 against 23.1, 2000 keys 19.4 against 14.6), unless the keys are few (26 x 60 tokens
  // over 60: 27 us with 32 rows, 20 with 16 and one wavefront).
  const auto cells = [&](int r) { return sequences * heads * ((rows + r - 1) / r); };
  p.wide = rows >= kWideRows && sequences == 1 && cells(kWideRows) * ones >= 7 * 256;
  p.group_rows = p.wide ? kWideRows : rows > 16 && keys > kFewKeys && cells(16) * ones > 20 * 256 ? 32 : 16;
  p.row_groups = (int)((rows + p.group_rows - 1) / p.group_rows);
  p.cells = cells(p.group_rows);
  // two workgroups to a CU where there are fewer cells (30000 tokens, 64 heads over 8: 21 us; 25 with four)
  int64_t splits = (512 + p.cells - 1) / p.cells;
  if (splits < (keys + kMaxChunk - 1) / kMaxChunk) splits = (keys + kMaxChunk - 1) / kMaxChunk;
  // Up to four steps of the four wavefronts stay in one chunk, since a join costs more than two or three steps (300 keys in one chunk
  // and in three: one row of 32 heads 7.6 us and 7.7, 4 x 16 tokens of 8 x 8 heads 8.2 and 11.2), but for four steps of few cells
  // (511 keys of one row of 32 heads: 8.5 us in one chunk, 7.9 in four; 4 x 32 heads: 8.7, 9.3).  Longer chunks have two steps
  // or more (2000 keys of one row of 32 heads: 10.6 us in eight chunks, 11.2 in sixteen).
  const int64_t steps = ones <= 3 ? 3 : ones > 4 ? 2 : p.cells <= 64 ? 1 : 4;
  const int64_t most = (ones + steps - 1) / steps;
  if (splits > most) splits = most;
  if (splits > kMaxSplits) splits = kMaxSplits;
  const int64_t fit = kMaxParts / (p.cells * p.group_rows * (int64_t)(dim * sizeof(float) + sizeof(float2)));
  if (splits > fit) splits = fit > 1 ? fit : 1;
  p.chunk = (int)((((keys + splits - 1) / splits) + unit - 1) / unit * unit);
  p.splits = (int)((keys + p.chunk - 1) / p.chunk);
  // One wavefront where a cell is one block of keys, or where few keys meet more cells than the card holds workgroups of four:
  // a small workgroup's chain is as long as a large one's, and four times as many run (64 x 52 heads of one row: 100 keys 18 us
  // against 27, 250 keys of 60 x 52 17 against 22, but 1000 keys 92 against 82; 64 x 8 heads: 120 keys 9.1 against 8.3).
  p.waves = p.group_rows == 16 && p.splits == 1 && (keys <= kBlock || (p.cells > 1024 && keys <= kFewKeys)) ? 1 : kWaves;
  const size_t parts = p.splits > 1 ? (size_t)p.cells * p.splits * p.group_rows : 0;
  p.ml_bytes = parts * sizeof(float2);
  p.o_bytes = parts * dim * sizeof(float);
  p.joined_inline = !p.wide && p.splits > 1 && p.splits <= kInline && p.cells <= kMaxCells;
  p.need = parts ? kCounterBytes + p.ml_bytes + p.o_bytes : 0;
  return p;
}

template <int KIND, int D>
void launch(const AttnPlan& p, const AttnArgs& a, int sequences, hipStream_t s) {
  // Chunks vary slowest: workgroups go to the eight XCDs in turn, and the last chunks of a ragged batch are mostly
  // empty.  Row groups of a head, which read the same keys, meet on one XCD where heads are a multiple of 8.
  const dim3 grid(a.c.heads * p.row_groups, sequences, p.splits);
  if (p.wide)
    hipLaunchKernelGGL((tree_attention_wide_kernel<KIND, D>), grid, dim3(256), 0, s, a);
  else if (p.waves == 1)
    hipLaunchKernelGGL((tree_attention_kernel<KIND, D, 1, 1>), grid, dim3(64), 0, s, a);
  else if (p.group_rows == 16)
    hipLaunchKernelGGL((tree_attention_kernel<KIND, D, 1, kWaves>), grid, dim3(64 * kWaves), 0, s, a);
  else
    hipLaunchKernelGGL((tree_attention_kernel<KIND, D, 2, kWaves>), grid, dim3(64 * kWaves), 0, s, a);
  if (p.splits > 1 && !p.joined_inline)
    hipLaunchKernelGGL((tree_attention_join_kernel<D>), dim3((unsigned)p.cells, p.group_rows), dim3(256), 0, s, a, p.splits);
}

}  // namespace
}  // namespace cl

using namespace cl;

extern "C" size_t cl_tree_attention_work_bytes(int32_t sequences, int32_t q_heads, int32_t heads, int32_t dim,
                                               int32_t max_q, int32_t max_ctx) {
  if (sequences < 1 || heads < 1 || q_heads < heads || q_heads % heads || dim < 1 || max_q < 1 || max_ctx < 0) return 0;
  return plan_attention(sequences, q_heads, heads, dim, max_q, max_ctx).need;
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
  const AttnPlan p = plan_attention(sequences, q_heads, cache->heads, cache->dim, max_q, max_ctx);
  if (p.cells > 0x7FFFFFFF) return fail(CL_ESIZE, "attention: too many sequences and heads");
  if ((int64_t)cache->heads * p.row_groups > 65535) return fail(CL_ESIZE, "attention: too many heads and row groups");
  if (p.need && (!work || work_bytes < p.need))
    return fail(CL_ENOMEM, "attention: work has %zu bytes, %zu are needed", work_bytes, p.need);
  if (!aligned_to(work, 16)) return fail(CL_EINVAL, "attention: work must be 16-byte aligned");
  uint8_t* w = static_cast<uint8_t*>(work);
  AttnArgs a = {static_cast<const uint16_t*>(q), static_cast<uint16_t*>(o), *cache, block_table, ctx_lens, cu_q,
                reinterpret_cast<const uint64_t*>(mask), p.joined_inline ? reinterpret_cast<uint32_t*>(w) : nullptr,
                reinterpret_cast<float2*>(w + kCounterBytes),
                reinterpret_cast<float*>(w + kCounterBytes + p.ml_bytes),
                q_token, q_head, tokens, q_heads / cache->heads, table_width, max_q, mask_words, dtype == CL_BF16,
                p.chunk, p.row_groups, p.group_rows, __builtin_ctz(cache->page_size), scale};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (cache->kind == CL_KV_INT8) {
    if (cache->dim == 128)
      launch<CL_KV_INT8, 128>(p, a, sequences, s);
    else
      launch<CL_KV_INT8, 64>(p, a, sequences, s);
  } else {
    if (cache->dim == 128)
      launch<CL_KV_INT4, 128>(p, a, sequences, s);
    else
      launch<CL_KV_INT4, 64>(p, a, sequences, s);
  }
  return launched("attention");
}

extern "C" cl_status cl_recording(void* stream, uint64_t* id) {
  clear_error();
  if (!id) return fail(CL_EINVAL, "recording: a required pointer is NULL");
  hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
  unsigned long long n = 0;
  const hipError_t e = hipStreamGetCaptureInfo(static_cast<hipStream_t>(stream), &st, &n);
  if (e != hipSuccess) return fail(CL_EHIP, "recording: %s", hipGetErrorString(e));
  *id = st == hipStreamCaptureStatusNone ? 0 : n;
  return CL_OK;
}
