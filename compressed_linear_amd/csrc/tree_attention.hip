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
// over channels and keys in any order that both operands follow: K is read in 16-byte
// pieces of a key's channels, V in pieces of 8 channels of each of a lane's
// eight keys, which v_perm transposes while it widens the codes.
//
// Exactness: int8 codes are fp16 values (the byte as a subnormal, one packed fma
// makes it code * 2^-9), their scales go to the fp32 scores (K) and to the
// probabilities (V); int4 codes times their 8-bit scales are fp16 values.  Q is
// scaled per row by a power of two into fp16's range.  So the only rounding
// below fp32 is that of the probabilities to fp16: they are kept near 2^11 of
// fp16's range relative to the running maximum and the largest V scale.
//
// The running maximum moves only when a score passes it by 2^4 (one vote of the
// wavefront a step), so that the output is rarely rescaled.
//
// The keys of a sequence are cut into chunks, a workgroup each, whose four
// wavefronts take every fourth block of 32 keys; the partial outputs of more than one
// chunk are joined by a second, small launch.
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
constexpr float kNone = -3.4e38f;  // running maximum before any key
constexpr float kSlack = 4.f;      // log2 by which a score may pass the running maximum
constexpr int kProbBits = 11;      // probabilities are scaled by 2^11: with the slack at most 2^15

constexpr int kMaxSplits = 1024;   // chunks that a sequence's keys are cut into

struct AttnArgs {
  const uint16_t* q;
  uint16_t* o;
  cl_kv_cache c;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  const int32_t* cu_q;
  const uint64_t* mask;
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
  int64_t n, chunk;
};
__device__ __forceinline__ Range range_of(const AttnArgs& a, int b, int max_splits) {
  Range x;
  x.first = a.cu_q[b];
  const int64_t n_new = (int64_t)a.cu_q[b + 1] - x.first;
  x.n_new = x.first < 0 || n_new < 0 || n_new > a.max_q || x.first + n_new > a.tokens ? 0 : (int)n_new;
  x.ctx = max(a.ctx_lens[b], 0);
  x.n = (int64_t)x.ctx + x.n_new;
  const int64_t least = (x.n + max_splits - 1) / max_splits;
  x.chunk = least <= a.chunk ? a.chunk : (least + kBlock * kWaves - 1) / (kBlock * kWaves) * (kBlock * kWaves);
  x.splits = (int)((x.n + x.chunk - 1) / x.chunk);
  return x;
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

// Two bytes code + 128, as fp16 subnormals in the halves of a word -> code * 2^-9, exactly.
__device__ __forceinline__ uint32_t widen8(uint32_t pair) {
  const h2 a = __builtin_bit_cast(h2, pair);
  const h2 r = __builtin_elementwise_fma(a, h2{(_Float16)32768.f, (_Float16)32768.f}, h2{(_Float16)-0.25f, (_Float16)-0.25f});
  return __builtin_bit_cast(uint32_t, r);
}

// Nibbles `at` (0, 4, 8 or 12) of the two halves of a word -> (nibble - 8) * s, exactly (s of 8 significant bits).
__device__ __forceinline__ uint32_t widen4(uint32_t word, int at, h2 s) {
  const uint32_t n = ((word >> at) & 0x000F000Fu) | 0x64006400u;  // 1024 + nibble
  const h2 c = __builtin_bit_cast(h2, n) - h2{(_Float16)1032.f, (_Float16)1032.f};
  return __builtin_bit_cast(uint32_t, c * s);
}

// What a wavefront loads for one block of 32 keys.
template <int KIND, int D>
struct Block;

template <int D>
struct Block<CL_KV_INT8, D> {
  u4 k[2][D / 64];  // tile, piece: key l % 16, channels 64 piece + 16 (l / 16) ..
  u2 v[8];          // key 4 (l / 16) + i of either tile, channels (D / 16) (l % 16) ..  (D = 64: 4 channels, x only)
  u2 ks[2], vs[2];  // fp16 scales of keys 4 (l / 16) .. of either tile
};

template <int D>
struct Block<CL_KV_INT4, D> {
  u4 k[2];           // key l % 16, channels (D / 4) (l / 16) ..  (D = 64: 16 channels, x and y only)
  uint32_t v[8];     // key 4 (l / 16) + i, channels (D / 16) (l % 16) ..  (D = 64: 4 channels, the low half)
  uint16_t ks[2], vs[8];
};

// Channel of step s, slot j (0..7) of lane group g in the first product.
template <int KIND, int D>
__device__ __forceinline__ constexpr int q_channel(int s, int g) {
  return KIND == CL_KV_INT8 ? (s / 2) * 64 + 16 * g + (s % 2) * 8 : (D / 4) * g + 8 * s;
}

template <int KIND, int D, int RT>
__global__ void __launch_bounds__(256) tree_attention_kernel(AttnArgs a) {
  constexpr int STEPS = D / 32;  // matrix-core steps of a score tile
  constexpr int CB = D / 16;     // channel blocks of the output; lane c of a block's 16 rows is channel CB c + block
  constexpr int ROWS = 16 * RT, STRIDE = D + 4;
  __shared__ __align__(16) float s_o[kWaves][ROWS][STRIDE];
  __shared__ float2 s_ml[kWaves][ROWS];

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, c16 = l & 15, g = l >> 4;
  const int b = blockIdx.z, hk = blockIdx.y % a.c.heads, rg = blockIdx.y / a.c.heads;
  const Range range = range_of(a, b, gridDim.x);
  const int first = range.first, n_new = range.n_new, ctx = range.ctx, splits = range.splits, split = blockIdx.x;
  const int64_t n = range.n, chunk = range.chunk;
  const int G = a.group, rows = min(n_new * G - rg * ROWS, ROWS);  // rows of this workgroup that exist
  if (rows <= 0 || split >= splits) return;
  const int64_t k0 = split * chunk;
  const int blocks = (int)((min(n, k0 + chunk) - k0 + kBlock - 1) / kBlock);

  // ---- Q: rows n = l % 16 of each tile, scaled by a power of two, as the second operand
  uint32_t q[RT][STEPS][4];
  float rowc[RT];
  int tok[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = rg * ROWS + 16 * r + c16;
    tok[r] = row / G;
    const bool there = tok[r] < n_new;
    const uint16_t* qp = a.q + (int64_t)(first + (there ? tok[r] : 0)) * a.q_token + (int64_t)(hk * G + row % G) * a.q_head;
    float f[STEPS][8], top = 0.f;
    bool fine = true;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      u4 raw = {0, 0, 0, 0};
      if (there) raw = *reinterpret_cast<const u4*>(qp + q_channel<KIND, D>(s, g));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint16_t e = (uint16_t)(raw[j / 2] >> (16 * (j % 2)));
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
    rowc[r] = fmaxf(ldexpf(fabsf(a.scale) * 1.44269504f, e - 14 + (KIND == CL_KV_INT8 ? 9 : 0)), 1e-38f);
  }

  f4 o[RT][CB];
  float m[RT], sum[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = kNone;
    sum[r] = 0.f;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) o[r][cb] = f4{0.f, 0.f, 0.f, 0.f};
  }
  float vref = 0.f;  // a power of two above every V scale seen (int8)
  float vmul = 0.f;  // 2^kProbBits / vref

  const uint8_t* const kb = static_cast<const uint8_t*>(a.c.k);
  const uint8_t* const vb = static_cast<const uint8_t*>(a.c.v);
  const int tiles_shift = a.page_shift - 4;  // tiles of 16 keys in a page
  constexpr int ROWB = KIND == CL_KV_INT8 ? D : D / 2;
  constexpr int SC = KIND == CL_KV_INT8 ? 1 : D / 32;

  // pages of the wavefront's next 64 tiles, one to a lane: -1 outside the cache or the table, 0 for a tile past
  // the end (its keys are masked; page 0 is there to be read)
  int pages = 0;
  const auto load_pages = [&](int i) {
    const int64_t at = k0 + ((int64_t)(wave + kWaves * (i + (l >> 1))) * kBlock) + 16 * (l & 1);
    int p = 0;
    if (at < n) {
      const int64_t col = at >> a.page_shift;
      p = col < a.table_width ? a.block_table[(int64_t)b * a.table_width + col] : -1;
      if (p < 0 || p >= a.c.pages) p = -1;
    }
    pages = p;
  };
  // Loads step i's block; returns whether a tile of it has no page.
  const auto load = [&](int i, Block<KIND, D>& x) -> int {
    if ((i & 31) == 0) load_pages(i);
    int bad = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int page = __builtin_amdgcn_readlane(pages, 2 * (i & 31) + t);
      if (page < 0) bad |= 1 << t;
      const int tile = (int)((k0 + (int64_t)(wave + kWaves * i) * kBlock) >> 4) + t;
      const int64_t row = (((int64_t)max(page, 0) * a.c.heads + hk) << a.page_shift) + ((tile & ((1 << tiles_shift) - 1)) << 4);
      const uint8_t* kp = kb + row * ROWB;
      const uint8_t* vp = vb + row * ROWB;
      const uint16_t* ksp = a.c.k_scale + row * SC;
      const uint16_t* vsp = a.c.v_scale + row * SC;
      if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
        for (int p = 0; p < D / 64; ++p) x.k[t][p] = *reinterpret_cast<const u4*>(kp + c16 * ROWB + 64 * p + 16 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint8_t* at = vp + (4 * g + j) * ROWB + CB * c16;
          if constexpr (D == 128)
            x.v[4 * t + j] = *reinterpret_cast<const u2*>(at);
          else
            x.v[4 * t + j].x = *reinterpret_cast<const uint32_t*>(at);
        }
        x.ks[t] = *reinterpret_cast<const u2*>(ksp + 4 * g);
        x.vs[t] = *reinterpret_cast<const u2*>(vsp + 4 * g);
      } else {
        if constexpr (D == 128) {
          x.k[t] = *reinterpret_cast<const u4*>(kp + c16 * ROWB + 16 * g);
        } else {
          const u2 half = *reinterpret_cast<const u2*>(kp + c16 * ROWB + 8 * g);
          x.k[t].x = half.x, x.k[t].y = half.y;
        }
        x.ks[t] = ksp[c16 * SC + (D == 128 ? g : g / 2)];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint8_t* at = vp + (4 * g + j) * ROWB + CB / 2 * c16;
          if constexpr (D == 128)
            x.v[4 * t + j] = *reinterpret_cast<const uint32_t*>(at);
          else
            x.v[4 * t + j] = *reinterpret_cast<const uint16_t*>(at);
          x.vs[4 * t + j] = vsp[(4 * g + j) * SC + CB * c16 / 32];
        }
      }
    }
    return bad;
  };

  const int steps = wave < blocks ? (blocks - wave + kWaves - 1) / kWaves : 0;
  Block<KIND, D> cur, nxt;
  int bad = steps > 0 ? load(0, cur) : 0;
  for (int i = 0; i < steps; ++i) {
    const int bad_next = i + 1 < steps ? load(i + 1, nxt) : 0;
    const int64_t j0 = k0 + (int64_t)(wave + kWaves * i) * kBlock;
    const int left = (int)min(n - j0, (int64_t)kBlock);  // keys of the block that exist
    const bool special = j0 + kBlock > ctx || bad;       // some rows may not see some keys

    // ---- scores
    f4 s[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r) s[r][0] = s[r][1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        uint32_t k[4];
        if constexpr (KIND == CL_KV_INT8) {
          const u4 raw = cur.k[t][st / 2];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            k[j] = widen8(perm(0, raw[2 * (st % 2) + j / 2], j % 2 ? 0x0C030C02u : 0x0C010C00u));
        } else {
          const h2 ks = __builtin_bit_cast(h2, (uint32_t)cur.ks[t] * 0x10001u);
#pragma unroll
          for (int j = 0; j < 4; ++j) k[j] = widen4(cur.k[t][st], 4 * j, ks);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r][t] = mfma16(k, q[r][st], s[r][t]);
      }
    float vs[8];
    if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int sh = 16 * (j % 2);
        const float ks = Elem<CL_F16>::up((uint16_t)(cur.ks[j / 4][j % 4 / 2] >> sh));
        vs[j] = Elem<CL_F16>::up((uint16_t)(cur.vs[j / 4][j % 4 / 2] >> sh));
        const int key = 16 * (j / 4) + 4 * g + j % 4;
        if (special && key >= left) vs[j] = 0.f;  // no token there: the scale may be anything
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r][j / 4][j % 4] *= ks;
      }
    }
    if (special) {
      const int64_t rel = j0 - ctx;  // place of the block's first key among the new tokens
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        uint32_t see;  // keys of the block that the row sees
        if (!a.mask) {
          const int64_t cnt = tok[r] - rel + 1;
          see = cnt >= 32 ? ~0u : cnt <= 0 ? 0u : (1u << cnt) - 1u;
        } else if (rel <= -32) {
          see = ~0u;
        } else {
          const uint64_t* w = a.mask + (int64_t)(first + min(tok[r], n_new - 1)) * a.mask_words;
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
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = 16 * (j / 4) + 4 * g + j % 4;
          if (!((see >> key) & 1))
            s[r][j / 4][j % 4] = -INFINITY;
          else if ((bad >> (j / 4)) & 1)
            s[r][j / 4][j % 4] = __builtin_nanf("");
        }
      }
    }
    // ---- the running maximum, and the largest V scale
    float up[RT];
    bool move = false;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float t = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                      fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
      up[r] = t * rowc[r];
      move |= up[r] > m[r] + kSlack;
    }
    float vtop = 0.f;
    if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) vtop = fmaxf(vtop, vs[j]);
      move |= vtop > vref;
    }
    if (__any(move)) {
      float ratio = 1.f;
      if constexpr (KIND == CL_KV_INT8) {
        vtop = row_max(vtop);
        if (vtop > vref) {
          const float to = 2.f * __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, vtop) & 0x7F800000u);
          ratio = vref / to;
          vref = to;
          vmul = (float)(1 << kProbBits) / to;
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float top = fmaxf(m[r], row_max(up[r]));
        const float old = __builtin_amdgcn_exp2f(m[r] - top);
        m[r] = top;
        sum[r] *= old;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) o[r][cb] *= old * ratio;
      }
    }
    // ---- probabilities
    uint32_t p[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = s[r][j / 4][j % 4];
        e[j] = __builtin_amdgcn_exp2f(x * rowc[r] - m[r]);
        sum[r] += e[j];
        e[j] *= KIND == CL_KV_INT8 ? vs[j] * vmul : (float)(1 << kProbBits);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p[r][j] = __builtin_bit_cast(uint32_t, h2{(_Float16)e[2 * j], (_Float16)e[2 * j + 1]});
    }
    // ---- output
    if constexpr (KIND == CL_KV_INT8) {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        uint32_t v[4];
        const uint32_t sel = 0x0C040C00u + 0x00010001u * (cb % 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = widen8(perm(cur.v[2 * j + 1][cb / 4], cur.v[2 * j][cb / 4], sel));
#pragma unroll
        for (int r = 0; r < RT; ++r) o[r][cb] = mfma16(v, p[r], o[r][cb]);
      }
    } else {
      h2 sc[4];
      uint32_t lo[4], hi[4];  // channels 0..3 and 4..7 of two keys, one in each half
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t s0 = cur.vs[2 * j], s1 = cur.vs[2 * j + 1];
        if (special) {  // no token there: the scale may be anything
          const int key = 16 * (j / 2) + 4 * g + 2 * (j % 2);
          if (key >= left) s0 = 0;
          if (key + 1 >= left) s1 = 0;
        }
        sc[j] = __builtin_bit_cast(h2, s0 | s1 << 16);
        lo[j] = perm(cur.v[2 * j + 1], cur.v[2 * j], 0x05040100u);
        hi[j] = perm(cur.v[2 * j + 1], cur.v[2 * j], 0x07060302u);
      }
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = widen4(cb < 4 ? lo[j] : hi[j], 4 * (cb % 4), sc[j]);
#pragma unroll
        for (int r = 0; r < RT; ++r) o[r][cb] = mfma16(v, p[r], o[r][cb]);
      }
    }
    cur = nxt;
    bad = bad_next;
  }

  // ---- join the four wavefronts
  const float unit = KIND == CL_KV_INT8 ? 512.f / (float)(1 << kProbBits) * vref : 1.f / (float)(1 << kProbBits);
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float l_row = row_sum(sum[r]);
    const int row = 16 * r + c16;
    if (g == 0) s_ml[wave][row] = make_float2(m[r], l_row);
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
  for (int row = tid / PARTS; row < rows; row += 256 / PARTS) {
    float top = kNone, w[kWaves], den = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kWaves; ++v) top = fmaxf(top, s_ml[v][row].x);
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      w[v] = __builtin_amdgcn_exp2f(s_ml[v][row].x - top);
      den += w[v] * s_ml[v][row].y;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] += w[v] * s_o[v][row][ch + j];
    }
    if (splits == 1) {
      store(row, x, den == 0.f ? 0.f : 1.f / den);
    } else {
      const int64_t at = (cell * gridDim.x + split) * ROWS + row;
      if (ch == 0) a.part_ml[at] = make_float2(top, den);
      f4* po = reinterpret_cast<f4*>(a.part_o + at * D + ch);
      po[0] = f4{x[0], x[1], x[2], x[3]};
      po[1] = f4{x[4], x[5], x[6], x[7]};
    }
  }
}

// Joins the partial outputs of a row's chunks, in chunk order within each of eight strands and the strands in
// order: 32 lanes (dim 128) or 16 hold four channels each.  A launch of its own rather than the workgroup that
// finishes last: rows x chunks partials are read by as many workgroups as there are rows.
template <int D>
__global__ void __launch_bounds__(256) tree_attention_join_kernel(AttnArgs a, int max_splits) {
  constexpr int LANES = D / 4, STRANDS = 256 / LANES;
  __shared__ float s_w[kMaxSplits];
  __shared__ __align__(16) f4 s_x[STRANDS][LANES];
  __shared__ float s_red[2 * kWaves];
  const int tid = threadIdx.x, cell = blockIdx.x, row = blockIdx.y;
  const int rg = cell % a.row_groups, hk = cell / a.row_groups % a.c.heads, b = cell / a.row_groups / a.c.heads;
  const Range x = range_of(a, b, max_splits);
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
  int rt, row_groups, splits, chunk;
  int64_t cells;
  size_t ml_bytes, o_bytes, need;
};

AttnPlan plan_attention(int64_t sequences, int q_heads, int heads, int dim, int max_q, int64_t max_ctx) {
  AttnPlan p;
  const int64_t rows = (int64_t)max_q * (q_heads / heads);
  p.rt = rows > 16 ? 2 : 1;
  p.row_groups = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
  p.cells = sequences * heads * p.row_groups;
  const int64_t keys = max_ctx + max_q, unit = kBlock * kWaves;
  int64_t splits = (1024 + p.cells - 1) / p.cells;
  const int64_t most = (keys + unit - 1) / unit;
  if (splits > most) splits = most;
  p.chunk = (int)((((keys + splits - 1) / splits) + unit - 1) / unit * unit);
  p.splits = (int)((keys + p.chunk - 1) / p.chunk);
  const size_t parts = p.splits > 1 ? (size_t)p.cells * p.splits * 16 * p.rt : 0;
  p.ml_bytes = parts * sizeof(float2);
  p.o_bytes = parts * dim * sizeof(float);
  p.need = p.ml_bytes + p.o_bytes;
  return p;
}

template <int KIND, int D>
void launch(const AttnPlan& p, const AttnArgs& a, int sequences, hipStream_t s) {
  const dim3 grid(p.splits, a.c.heads * p.row_groups, sequences);
  if (p.rt == 1)
    hipLaunchKernelGGL((tree_attention_kernel<KIND, D, 1>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((tree_attention_kernel<KIND, D, 2>), grid, dim3(256), 0, s, a);
  if (p.splits > 1)
    hipLaunchKernelGGL((tree_attention_join_kernel<D>), dim3((unsigned)p.cells, 16 * p.rt), dim3(256), 0, s, a, p.splits);
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
                reinterpret_cast<const uint64_t*>(mask), reinterpret_cast<float2*>(w),
                reinterpret_cast<float*>(w + p.ml_bytes),
                q_token, q_head, tokens, q_heads / cache->heads, table_width, max_q, mask_words, dtype == CL_BF16,
                p.chunk, p.row_groups, 16 * p.rt, __builtin_ctz(cache->page_size), scale};
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
