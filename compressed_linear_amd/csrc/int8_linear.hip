// int8_linear.hip -- the linear layer in 8-bit integers: rows of values to codes with a scale each, and the product
// of two sets of such rows.
#include <algorithm>

#include "cl_int8.h"
#include "int8_plan.h"
#include "serving.h"

namespace cl {
namespace {

constexpr int kMostK = 131071;  // 128 * 128 * K < 2^31
constexpr int kMostN = 1 << 25;
constexpr int64_t kMostRow = 1 << 23;  // 256 rows of it are within 32 bits
constexpr float kLeast = 0x1p-100f;

// A value as it is quantised: clamped where there is a clamp (a NaN stays one).
__device__ __forceinline__ float clamped(float v, float clamp) { return clamp > 0.f && fabsf(v) > clamp ? copysignf(clamp, v) : v; }

// ------------------------------------------------------------------- codes
// Eight values of a row from k on, as they are quantised; zeros past its end.  Rows may lie at any multiple of an element: the hardware
// takes loads of 16 bytes there.
template <int IN>
__device__ __forceinline__ void values8(const typename Elem<IN>::raw* x, int k, int K, float clamp, float (&v)[8]) {
  if (k + 8 <= K) {
    typename Elem<IN>::raw some[8];
    __builtin_memcpy(some, x + k, sizeof some);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<IN>::up(some[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (k < K) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (k + i < K) v[i] = Elem<IN>::up(x[k + i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = clamped(v[i], clamp);
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

// A row's scale and its inverse, from its largest magnitude as bits (those of a NaN or an infinity are larger than a number's).
struct RowScale {
  float scale, inverse;
};
__device__ __forceinline__ RowScale row_scale(uint32_t most) {
  const float a = __builtin_bit_cast(float, most);
  if (most >= 0x7f800000u) return {__builtin_nanf(""), 0.f};
  if (a < kLeast) return {0.f, 0.f};
  const float s = a * (1.f / 127.f);
  return {s, 1.f / s};
}

// Eight codes in two words.  |v| (1 / s) passes 127 by its roundings only, which rint takes away; an inverse of 0 gives 0 whatever v is.
__device__ __forceinline__ w2 codes8(const float (&v)[8], float inverse) {
  w2 w = {0, 0};
  if (inverse == 0.f) return w;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i / 4] |= ((uint32_t)(int)rintf(v[i] * inverse) & 255) << (8 * (i % 4));
  return w;
}

// A workgroup a row, eight values to a thread at a time, the first HELD of them kept in registers between the two passes.
// Bound by memory, few rows by the two trips to it.
template <int IN, int THREADS, int HELD>
__global__ void __launch_bounds__(THREADS) int8_quant_kernel(const typename Elem<IN>::raw* __restrict__ x, int64_t x_row, int64_t first, int K, int width,
                                                             float clamp, int8_t* __restrict__ codes, int64_t row, float* __restrict__ scale) {
  __shared__ uint32_t most[THREADS / 64];
  const int64_t t = first + blockIdx.x;
  x += t * x_row;
  float held[HELD][8];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < HELD; ++c) {
    values8<IN>(x, 8 * (c * THREADS + threadIdx.x), K, clamp, held[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, magnitude(held[c][i]));
  }
  for (int k = 8 * (HELD * THREADS + threadIdx.x); k < K; k += 8 * THREADS) {
    float v[8];
    values8<IN>(x, k, K, clamp, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[i]));
  }
#pragma unroll
  for (int d = 32; d; d /= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) m = max(m, most[w]);
  }
  const RowScale s = row_scale(m);
  if (threadIdx.x == 0) scale[t] = s.scale;
  w2* to = reinterpret_cast<w2*>(codes + t * row);
#pragma unroll
  for (int c = 0; c < HELD; ++c) {
    const int k = 8 * (c * THREADS + threadIdx.x);
    if (k < width) to[k / 8] = codes8(held[c], s.inverse);
  }
  for (int k = 8 * (HELD * THREADS + threadIdx.x); k < width; k += 8 * THREADS) {
    float v[8];
    values8<IN>(x, k, K, clamp, v);
    to[k / 8] = codes8(v, s.inverse);
  }
}

// ----------------------------------------------------------------- product
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i16x __attribute__((ext_vector_type(16)));

constexpr int kSums = 3;  // an output type past cl_dtype's: the sums themselves, of a part of K

// What a product works on.  Sums of a part of K go to `sums` [parts, tokens, pitch], whose rows are a multiple of 4.
struct Product {
  const int8_t* codes;
  int64_t row;
  const float* scale;
  int tokens;
  const int8_t* w;
  int64_t w_row;
  const float *w_scale, *bias;
  int N, steps;  // K in steps of 128
  void* y;
  int64_t y_row;
  int32_t* sums;
  int pitch;
};

template <int OUT>
struct Result {
  typedef typename Elem<OUT>::raw raw;
};
template <>
struct Result<kSums> {
  typedef int32_t raw;
};

// Each product and the sum rounded to fp32 (no fused multiply-add), so that every kernel gives a row the same bits.
__device__ __forceinline__ float scaled(const Product& p, int sum, float s, int n) {
#pragma clang fp contract(off)
  const float v = (float)sum * s * p.w_scale[n];
  return p.bias ? v + p.bias[n] : v;
}

// Waits until at most N loads are under way, those into LDS among them.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt has six bits");
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | N >> 4 << 14);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}
__device__ __forceinline__ void wait_lds() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}
__device__ __forceinline__ void meet() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// A tile of TW outputs by TT tokens, by GW x GT wavefronts of FW x FT blocks of 32 x 32 (v_mfma_i32_32x32x32_i8, weights as
// the first operand, so that a lane has four outputs side by side of one token).  Steps of 128 k: the rows' 128 bytes come into LDS
// directly, DEPTH - 1 steps ahead, into a ring of DEPTH buffers; a row's eight pieces of 16 bytes lie permuted by (row / 2) % 8, so that the 16
// lanes which LDS serves at once read all its banks.  A quarter step's operands are read between the products of the one before.  The
// one barrier of a step stands before its last quarter, whose operands are in registers: behind it the next buffer has arrived
// everywhere and this one is read by nobody.  Rows past the last and steps past the end are not read (the loads know their buffer's size), and
// what LDS holds in their place reaches no output.  ONCE: the weights are not kept in the caches, since no other tile reads them.
// Bound by waiting for memory and, where there are many tiles, by power too (2048 x 8192 x 28672, 417 us, 2.31 POPS launch after launch:
// the matrix cores busy 60 % of the cycles, the clock at 1.83 of 2.4 GHz; with codes of zeros 367 us, 52 % at 2.41 GHz, so that power costs an
// eighth and waiting the rest).
template <int OUT, int TW, int TT, int GW, int GT, int DEPTH, bool ONCE>
__device__ __forceinline__ void tile(const Product& p, uint8_t* lds, int t0, int n0, int first, int end, int part) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int WAVES = GW * GT, FW = TW / GW / 32, FT = TT / GT / 32, ROWS = TW + TT, STAGE = ROWS * 128;
  constexpr int LOADS = ROWS / 8 / WAVES;  // loads of a wavefront for a step, 8 rows each
  static_assert(TW % (8 * WAVES) == 0 && TT % (8 * WAVES) == 0, "a wavefront's loads are weights or tokens");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int8_t* w_base = p.w + (int64_t)n0 * p.w_row;
  const int8_t* t_base = p.codes + (int64_t)t0 * p.row;
  const uint32_t w_bytes = (uint32_t)(min(TW, p.N - n0) * p.w_row), t_bytes = (uint32_t)(min(TT, p.tokens - t0) * p.row);
  uint32_t at_row[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = (i * WAVES + wave) * 8 + (lane >> 3), piece = (lane & 7) ^ ((r >> 1) & 7);
    at_row[i] = (i * WAVES * 8 < TW ? (uint32_t)(r * p.w_row) : (uint32_t)((r - TW) * p.row)) + piece * 16;
  }
  const auto load = [&](int step, int buf) {
    const bool any = step < end;
    const auto w = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(w_base), 0, any ? w_bytes : 0, 0x00020000);
    const auto t = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(t_base), 0, any ? t_bytes : 0, 0x00020000);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      auto to = (__attribute__((address_space(3))) void*)(lds + buf * STAGE + (i * WAVES + wave) * 1024);
      if (i * WAVES * 8 < TW)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(w, to, 16, at_row[i], step * 128, 0, ONCE ? 2 : 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(t, to, 16, at_row[i], step * 128, 0, 0);
    }
  };
  const int ww = wave % GW, wt = wave / GW, r = lane & 31, half = lane >> 5;
  const uint8_t* w_at = lds + (ww * FW * 32 + r) * 128;
  const uint8_t* t_at = lds + (TW + wt * FT * 32 + r) * 128;
  uint32_t at_piece[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) at_piece[q] = ((2 * q + half) ^ ((r >> 1) & 7)) * 16;
  i4 fw[2][FW], ft[2][FT];
  i16x acc[FW][FT] = {};
  const auto read = [&](int buf, int quarter, int to) {
    const uint32_t at = at_piece[quarter] + buf * STAGE;
#pragma unroll
    for (int i = 0; i < FW; ++i) fw[to][i] = *reinterpret_cast<const i4*>(w_at + i * 4096 + at);
#pragma unroll
    for (int j = 0; j < FT; ++j) ft[to][j] = *reinterpret_cast<const i4*>(t_at + j * 4096 + at);
  };
  const auto multiply = [&](int of) {
#pragma unroll
    for (int i = 0; i < FW; ++i)
#pragma unroll
      for (int j = 0; j < FT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[of][i], ft[of][j], acc[i][j], 0, 0, 0);
  };
  // the order of a quarter: a read, a load and a product in turn
  const auto mix = [&](int loads) {
    constexpr int READS = FW + FT, PRODUCTS = FW * FT, MOST = READS > PRODUCTS ? READS : PRODUCTS;
#pragma unroll
    for (int i = 0; i < (MOST > LOADS ? MOST : LOADS); ++i) {
      if (i < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (i < loads) __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
      if (i < PRODUCTS) __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    }
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(first + d, d);
  wait_loads<(DEPTH - 1) * LOADS>();
  meet();
  read(0, 0, 0);
  for (int at = first, buf = 0; at < end; ++at) {
    const int next = DEPTH == 2 ? buf ^ 1 : buf + 1 == DEPTH ? 0 : buf + 1;
    read(buf, 1, 1);
    multiply(0);
    mix(0);
    read(buf, 2, 0);
    multiply(1);
    mix(0);
    read(buf, 3, 1);
    multiply(0);
    mix(0);
    wait_lds();
    wait_loads<(DEPTH - 2) * LOADS>();
    meet();
    load(at + DEPTH, buf);
    read(next, 0, 0);
    multiply(1);
    mix(LOADS);
    buf = next;
  }
  wait_lds();
  wait_loads<0>();
  meet();
  // Out through LDS, 32 tokens of a wavefront at a time, so that rows are written in pieces of 16 bytes.
  typedef typename Result<OUT>::raw raw;
  constexpr int PITCH = FW * 32 * sizeof(raw) + 16, PER = 16 / sizeof(raw), ACROSS = FW * 32 / PER, DOWN = 64 / ACROSS;
  uint8_t* mine = lds + wave * (32 * PITCH);
  const int nb = n0 + ww * FW * 32;
  raw* y = OUT == kSums ? reinterpret_cast<raw*>(p.sums) + (int64_t)part * p.tokens * p.pitch : static_cast<raw*>(p.y);
  const int64_t y_row = OUT == kSums ? p.pitch : p.y_row;
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const int tb = t0 + (wt * FT + j) * 32;
    const float s = OUT == kSums ? 0.f : p.scale[min(tb + r, p.tokens - 1)];
#pragma unroll
    for (int i = 0; i < FW; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = i * 32 + 8 * q + 4 * half;
        uint8_t* to = mine + r * PITCH + n * sizeof(raw);
        if constexpr (OUT == kSums) {
          *reinterpret_cast<i4*>(to) = i4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        } else {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = scaled(p, acc[i][j][4 * q + e], s, min(nb + n + e, p.N - 1));
          if constexpr (OUT == CL_F32)
            *reinterpret_cast<v4*>(to) = v4{v[0], v[1], v[2], v[3]};
          else
            *reinterpret_cast<w2*>(to) = w2{down2<OUT>(v[0], v[1]), down2<OUT>(v[2], v[3])};
        }
      }
    wait_lds();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < 32 / DOWN; ++k) {
      const int down = k * DOWN + lane / ACROSS, across = lane % ACROSS * PER, t = tb + down, n = nb + across;
      if (t >= p.tokens || n >= p.N) continue;
      raw v[PER];
      *reinterpret_cast<w4*>(v) = *reinterpret_cast<const w4*>(mine + down * PITCH + across * sizeof(raw));
      if (OUT == kSums || n + PER <= p.N) {
        __builtin_memcpy(y + t * y_row + n, v, sizeof v);  // at any multiple of an element
      } else {
#pragma unroll
        for (int e = 0; e < PER; ++e)
          if (n + e < p.N) y[t * y_row + n + e] = v[e];
      }
    }
    wait_lds();
    __builtin_amdgcn_sched_barrier(0);
  }
#endif
}

// Tiles in runs of eight token tiles, those first, then the next outputs: what the 32 workgroups of an XCD read at a time are rows of few
// tiles, and the XCDs (workgroup number % 8) have runs of their own.
struct Tiles {
  int t, w, parts;  // tiles along the tokens and the outputs, parts of K
  int full;         // tiles of the whole size; behind them come halves of tiles (half the tokens)
};
__device__ __forceinline__ int of_xcd(int id, int n) {
  const int xcd = id & 7, each = n >> 3, extra = n & 7;
  return xcd * each + min(xcd, extra) + (id >> 3);
}
// The rings' rows of 128 bytes, or 32 rows of each wavefront's outputs.
constexpr int lds_bytes(int rows, int half_rows, int waves, int out) {
  const int ring = 128 * (rows > half_rows ? rows : half_rows), outputs = waves * 32 * (out + 16);
  return ring > outputs ? ring : outputs;
}
template <int OUT, int TW, int TT, int GW, int GT, int DEPTH, bool HALVES, bool ONCE>
__global__ void __launch_bounds__(64 * GW * GT, 2) int8_tile_kernel(Product p, Tiles g) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[lds_bytes((TW + TT) * DEPTH, (TW + TT / 2) * (HALVES ? DEPTH + 1 : 0), GW * GT,
                                                                 TW / GW * (int)sizeof(typename Result<OUT>::raw))];
  const bool half = HALVES && (int)blockIdx.x >= g.full;
  const int unit = half ? of_xcd(blockIdx.x - g.full, gridDim.x - g.full) : of_xcd(blockIdx.x, HALVES ? g.full : gridDim.x);
  const int tiles = g.t * g.w, at = half ? g.full + (unit >> 1) : unit, part = at / tiles, number = at % tiles;
  const int run = number / (8 * g.w), in = number % (8 * g.w), high = min(8, g.t - 8 * run);
  const int t0 = (8 * run + in % high) * TT, n0 = in / high * TW;
  const int first = (int)((int64_t)p.steps * part / g.parts), end = (int)((int64_t)p.steps * (part + 1) / g.parts);
  if constexpr (HALVES) {
    if (half) {
      const int t = t0 + (unit & 1) * (TT / 2);
      if (t < p.tokens) tile<OUT, TW, TT / 2, GW, GT, DEPTH + 1, ONCE>(p, lds, t, n0, first, end, part);
      return;
    }
  }
  tile<OUT, TW, TT, GW, GT, DEPTH, ONCE>(p, lds, t0, n0, first, end, part);
}

// Sums of parts of K to outputs, four to a thread.
template <int OUT>
__global__ void __launch_bounds__(256) int8_join_kernel(Product p, int parts, int64_t first) {
  const int64_t at = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int across = p.pitch / 4, n = 4 * (int)(at % across);
  const int64_t t = at / across;
  if (t >= p.tokens) return;
  i4 sum = {0, 0, 0, 0};
  for (int k = 0; k < parts; ++k) sum += *reinterpret_cast<const i4*>(p.sums + (k * (int64_t)p.tokens + t) * p.pitch + n);
  const float s = p.scale[t];
  typename Elem<OUT>::raw* y = static_cast<typename Elem<OUT>::raw*>(p.y) + t * p.y_row + n;
  typename Elem<OUT>::raw v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = Elem<OUT>::down(scaled(p, sum[e], s, min(n + e, p.N - 1)));
  if (n + 4 <= p.N) {
    __builtin_memcpy(y, v, sizeof v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) y[e] = v[e];
  }
}

// ------------------------------------------------------------- few tokens
// Few tokens: the weights are read once, which bounds it (one token of 8192 x 28672 37.5 us, 6.3 TB/s).  A workgroup has 16 outputs; its wavefronts take the steps of 128 k in turn, each with a
// ring of DEPTH buffers in LDS to itself, so that they wait for their own loads only, and their sums meet in LDS at the end
// (v_mfma_i32_16x16x64_i8, weights as the first operand).  Rows lie as in a tile; TR (8, or a multiple of 16) token rows come with the weights.
template <int OUT, int WAVES, int DEPTH, int TR>
__global__ void __launch_bounds__(64 * WAVES) int8_stream_kernel(Product p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int LOADS = (16 + TR) / 8, STAGE = (16 + TR) * 128, FT = (TR + 15) / 16;
  __shared__ __attribute__((aligned(128))) uint8_t ring[WAVES][DEPTH][STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = blockIdx.x * 16;
  const int8_t* w_base = p.w + (int64_t)n0 * p.w_row;
  const uint32_t w_bytes = (uint32_t)(min(16, p.N - n0) * p.w_row), t_bytes = (uint32_t)(p.tokens * p.row);
  uint32_t at_row[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = i * 8 + (lane >> 3), piece = (lane & 7) ^ ((r >> 1) & 7);
    at_row[i] = (i < 2 ? (uint32_t)(r * p.w_row) : (uint32_t)((r - 16) * p.row)) + piece * 16;
  }
  const auto load = [&](int step, int buf) {
    const bool any = step < p.steps;
    const auto w = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(w_base), 0, any ? w_bytes : 0, 0x00020000);
    const auto t = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p.codes), 0, any ? t_bytes : 0, 0x00020000);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      auto to = (__attribute__((address_space(3))) void*)(ring[wave][buf] + i * 1024);
      if (i < 2)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(w, to, 16, at_row[i], step * 128, 0, 2);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(t, to, 16, at_row[i], step * 128, 0, 0);
    }
  };
  const int r = lane & 15, q = lane >> 4, tr = 16 + (TR == 8 ? r & 7 : r);
  uint32_t w_at[2], t_at[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w_at[h] = r * 128 + ((q + 4 * h) ^ ((r >> 1) & 7)) * 16;
    t_at[h] = tr * 128 + ((q + 4 * h) ^ ((tr >> 1) & 7)) * 16;
  }
  i4 acc[2][FT] = {};
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(wave + d * WAVES, d);
  for (int step = wave, buf = 0; step < p.steps; step += WAVES) {
    wait_loads<(DEPTH - 1) * LOADS>();
    const uint8_t* at = ring[wave][buf];
    i4 fw[2], ft[2][FT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      fw[h] = *reinterpret_cast<const i4*>(at + w_at[h]);
#pragma unroll
      for (int j = 0; j < FT; ++j) ft[h][j] = *reinterpret_cast<const i4*>(at + t_at[h] + j * 2048);
    }
    wait_lds();
    load(step + DEPTH * WAVES, buf);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < FT; ++j) acc[h][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[h], ft[h][j], acc[h][j], 0, 0, 0);
    buf = buf + 1 == DEPTH ? 0 : buf + 1;
  }
  wait_loads<0>();
#pragma unroll
  for (int j = 0; j < FT; ++j) *reinterpret_cast<i4*>(ring[wave][0] + j * 1024 + lane * 16) = acc[0][j] + acc[1][j];
  __syncthreads();
  // a lane of a block's sums has outputs 4 (lane / 16) to + 3 of token lane % 16; a thread takes one at a time
  for (int k = threadIdx.x; k < FT * 256; k += 64 * WAVES) {
    const int j = k >> 8, t = k >> 4 & 15, n = k & 15;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += *reinterpret_cast<const int*>(ring[w][0] + j * 1024 + ((n >> 2) * 16 + t) * 16 + (n & 3) * 4);
    if (16 * j + t < p.tokens && n0 + n < p.N)
      static_cast<typename Elem<OUT>::raw*>(p.y)[(16 * j + t) * p.y_row + n0 + n] = Elem<OUT>::down(scaled(p, sum, p.scale[16 * j + t], n0 + n));
  }
#endif
}

cl_status check_weights(const int8_t* w, int64_t w_row, const float* w_scale, const float* bias, int N, int K) {
  if (N < 1 || K < 1) return fail(CL_EINVAL, "int8: N >= 1 and K >= 1 are wanted");
  if (K > kMostK) return fail(CL_ESIZE, "int8: K %d above %d", K, kMostK);
  if (N > kMostN) return fail(CL_ESIZE, "int8: N %d above %d", N, kMostN);
  if (!w || !w_scale) return fail(CL_EINVAL, "int8: w or w_scale is NULL");
  if (!aligned_to(w, 16) || !aligned_to(w_scale, 4) || (bias && !aligned_to(bias, 4)))
    return fail(CL_EINVAL, "int8: w must be 16-byte aligned, scales and bias 4-byte");
  if (w_row % 128 || w_row < K) return fail(CL_EINVAL, "int8: rows of %lld bytes for %d codes (a multiple of 128 is wanted)", (long long)w_row, K);
  if (w_row > kMostRow) return fail(CL_ESIZE, "int8: rows of more than %lld bytes", (long long)kMostRow);
  return CL_OK;
}

cl_status check_codes(const int8_t* codes, int64_t row, const float* scale, int K) {
  if (!codes || !scale) return fail(CL_EINVAL, "int8: codes or scale is NULL");
  if (!aligned_to(codes, 16) || !aligned_to(scale, 4)) return fail(CL_EINVAL, "int8: codes must be 16-byte aligned, scales 4-byte");
  if (row % 128 || row < K) return fail(CL_EINVAL, "int8: rows of %lld bytes for %d codes (a multiple of 128 is wanted)", (long long)row, K);
  if (row > kMostRow) return fail(CL_ESIZE, "int8: rows of more than %lld bytes", (long long)kMostRow);
  return CL_OK;
}

cl_status check_work(const void* work, size_t bytes, size_t need) {
  if (bytes < need) return fail(CL_ENOMEM, "int8: the workspace has %zu bytes, %zu are wanted", bytes, need);
  if (need && (!work || !aligned_to(work, 16))) return fail(CL_EINVAL, "int8: work is NULL or misaligned");
  return CL_OK;
}

Product product_of(const int8_t* codes, int64_t row, const float* scale, int tokens, const int8_t* w, int64_t w_row, const float* w_scale,
                   const float* bias, int N, int K, void* y, int64_t y_row, void* sums) {
  return {codes, row, scale, tokens, w, w_row, w_scale, bias, N, (int)(padded(K) / 128), y, y_row, static_cast<int32_t*>(sums), (N + 3) / 4 * 4};
}

cl_status check_output(const void* y, int y_dtype) {
  if (!elem_ok(y_dtype)) return fail(CL_EINVAL, "int8: unknown element type of y");
  if (!y || !aligned_to(y, elem_size(y_dtype))) return fail(CL_EINVAL, "int8: y is NULL or misaligned for its type");
  return CL_OK;
}

cl_status check_values(const void* x, int dtype, int K, float clamp) {
  if (K < 1) return fail(CL_EINVAL, "int8: K >= 1 is wanted");
  if (K > kMostK) return fail(CL_ESIZE, "int8: K %d above %d", K, kMostK);
  if (!elem_ok(dtype)) return fail(CL_EINVAL, "int8: unknown element type of x");
  if (!x || !aligned_to(x, elem_size(dtype))) return fail(CL_EINVAL, "int8: x is NULL or misaligned for its type");
  if (!(clamp >= 0.f) || !(clamp < __builtin_inff())) return fail(CL_EINVAL, "int8: clamp must be finite and >= 0");
  return CL_OK;
}

template <int IN, int THREADS, int HELD>
void launch_quant(const void* x, int64_t x_row, int rows, int K, float clamp, int8_t* codes, int64_t row, float* scale, hipStream_t s) {
  in_pieces(rows, THREADS, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL((int8_quant_kernel<IN, THREADS, HELD>), dim3((unsigned)count), dim3(THREADS), 0, s, static_cast<const typename Elem<IN>::raw*>(x), x_row, first, K,
                       (int)padded(K), clamp, codes, row, scale);
  });
}

// Rows of up to 8192 values are 8 or 16 to a thread, so that as many threads as can be ask for them (2048 rows of 8192 bf16 12.0 us with 512
// threads, 13.0 with 256 and with 1024, whose waits for each other cost more; of 4096 7.1 with 256 and 7.0 with 512); longer ones 1024 threads' registers up to
// 32768.
template <int IN>
void launch_quant(const void* x, int64_t x_row, int rows, int K, float clamp, int8_t* codes, int64_t row, float* scale, hipStream_t s) {
  if (K <= 2048)
    launch_quant<IN, 256, 1>(x, x_row, rows, K, clamp, codes, row, scale, s);
  else if (K <= 4096)
    launch_quant<IN, 256, 2>(x, x_row, rows, K, clamp, codes, row, scale, s);
  else if (K <= 8192)
    launch_quant<IN, 512, 2>(x, x_row, rows, K, clamp, codes, row, scale, s);
  else
    launch_quant<IN, 1024, 4>(x, x_row, rows, K, clamp, codes, row, scale, s);
}

void launch_quant(const void* x, int dtype, int64_t x_row, int rows, int K, float clamp, int8_t* codes, int64_t row, float* scale, hipStream_t s) {
  if (dtype == CL_F16)
    launch_quant<CL_F16>(x, x_row, rows, K, clamp, codes, row, scale, s);
  else if (dtype == CL_BF16)
    launch_quant<CL_BF16>(x, x_row, rows, K, clamp, codes, row, scale, s);
  else
    launch_quant<CL_F32>(x, x_row, rows, K, clamp, codes, row, scale, s);
}

// ------------------------------------------------------------------- launches
size_t sums_bytes(int tokens, int N, int K) {
  if (streamed(tokens, N, K)) return 0;
  const Plan p = plan_product(tokens, N, K);
  return p.parts > 1 ? (size_t)4 * p.parts * tokens * ((N + 3) / 4 * 4) : 0;
}

template <int OUT, int TW, int TT, int GW, int GT, int DEPTH, bool HALVES, bool ONCE>
void launch_tiles(const Product& p, int parts, hipStream_t s) {
  Tiles g{(p.tokens + TT - 1) / TT, (p.N + TW - 1) / TW, parts, 0};
  const int n = g.t * g.w * parts, rest = n % kCus;
  g.full = n;
  int blocks = n;
  if (HALVES && halved(n)) g.full = n - rest, blocks = g.full + 2 * rest;
  const auto kernel = int8_tile_kernel<OUT, TW, TT, GW, GT, DEPTH, HALVES, ONCE>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * GW * GT), 0, s, p, g);
}

template <int OUT>
void launch_shape(const Product& p, const Plan& plan, hipStream_t s) {
  switch (plan.shape) {
    case 0: return launch_tiles<OUT, 256, 256, 4, 2, 2, true, false>(p, plan.parts, s);
    case 1: return launch_tiles<OUT, 256, 192, 4, 2, 2, false, false>(p, plan.parts, s);
    case 2: return launch_tiles<OUT, 256, 128, 4, 2, 3, false, false>(p, plan.parts, s);
    case 3: return launch_tiles<OUT, 128, 128, 4, 2, 4, false, false>(p, plan.parts, s);
    case 4: return launch_tiles<OUT, 128, 64, 4, 2, 3, false, true>(p, plan.parts, s);
    case 5: return launch_tiles<OUT, 64, 64, 2, 2, 4, false, true>(p, plan.parts, s);
    default: return launch_tiles<OUT, 64, 32, 2, 1, 4, false, true>(p, plan.parts, s);
  }
}

template <int OUT, int WAVES, int DEPTH, int TR>
void launch_stream(const Product& p, hipStream_t s) {
  hipLaunchKernelGGL((int8_stream_kernel<OUT, WAVES, DEPTH, TR>), dim3((unsigned)((p.N + 15) / 16)), dim3(64 * WAVES), 0, s, p);
}

// Tokens past what a launch holds (2^22 tiles of 512 threads) go in pieces, which have tiles enough without parts of K.
template <int OUT>
void launch_linear(const Product& p, int K, hipStream_t s) {
  // eight wavefronts with three buffers: one token of 8192 x 10240 15.6 us, four 16.9, with four buffers 16.5, sixteen 18.5; with more
  // token rows two buffers (16 tokens of 8192 x 28672 41.4 us, three 48.7) and four wavefronts (32 tokens of 4096 x 11008 14.6, eight 17.5)
  if (p.tokens <= 8) return launch_stream<OUT, 8, 3, 8>(p, s);
  if (p.tokens <= 16) return launch_stream<OUT, 8, 2, 16>(p, s);
  if (streamed(p.tokens, p.N, K)) return p.tokens <= 32 ? launch_stream<OUT, 4, 2, 32>(p, s) : launch_stream<OUT, 4, 2, 64>(p, s);
  const Plan plan = plan_product(p.tokens, p.N, K);
  if (plan.parts > 1) {
    launch_shape<kSums>(p, plan, s);
    in_pieces((int64_t)p.tokens * (p.pitch / 4), 1, [&](int64_t first, int64_t count) {
      hipLaunchKernelGGL((int8_join_kernel<OUT>), dim3((unsigned)((count + 255) / 256)), dim3(256), 0, s, p, plan.parts, first);
    });
    return;
  }
  const int64_t most = std::max<int64_t>(1, (1 << 22) / ((p.N + 127) / 128) / 16) * 2048;
  for (int64_t first = 0; first < p.tokens; first += most) {
    Product q = p;
    q.codes += first * p.row;
    q.scale += first;
    q.y = beyond(p.y, OUT, first * p.y_row);
    q.tokens = (int)std::min(most, p.tokens - first);
    launch_shape<OUT>(q, plan, s);
  }
}

void launch_linear(const Product& p, int K, int out, hipStream_t s) {
  if (out == CL_F16)
    launch_linear<CL_F16>(p, K, s);
  else if (out == CL_BF16)
    launch_linear<CL_BF16>(p, K, s);
  else
    launch_linear<CL_F32>(p, K, s);
}

}  // namespace
}  // namespace cl

using namespace cl;

extern "C" size_t cl_int8_work_bytes(int32_t tokens, int32_t N, int32_t K, int32_t quantised) {
  if (tokens < 1 || N < 1 || N > kMostN || K < 1 || K > kMostK) return 0;
  return sums_bytes(tokens, N, K) + (quantised ? 0 : (size_t)tokens * (padded(K) + 4));
}

extern "C" cl_status cl_int8_quant(const void* x, int32_t dtype, int64_t x_row, int32_t rows, int32_t K, float clamp,
                                   int8_t* codes, int64_t row, float* scale, void* stream) {
  clear_error();
  if (rows < 0) return fail(CL_EINVAL, "int8: rows must be >= 0");
  if (rows == 0) return CL_OK;
  cl_status st = check_values(x, dtype, K, clamp);
  if (st == CL_OK) st = check_codes(codes, row, scale, K);
  if (st != CL_OK) return st;
  launch_quant(x, dtype, x_row, rows, K, clamp, codes, row, scale, static_cast<hipStream_t>(stream));
  return launched("int8 quant");
}

extern "C" cl_status cl_int8_linear(const int8_t* codes, int64_t row, const float* scale, int32_t tokens, const int8_t* w,
                                    int64_t w_row, const float* w_scale, const float* bias, int32_t N, int32_t K, void* y,
                                    int32_t y_dtype, int64_t y_row, void* work, size_t work_bytes, void* stream) {
  clear_error();
  if (tokens < 0) return fail(CL_EINVAL, "int8: tokens must be >= 0");
  if (tokens == 0) return CL_OK;
  cl_status st = check_weights(w, w_row, w_scale, bias, N, K);
  if (st == CL_OK) st = check_codes(codes, row, scale, K);
  if (st == CL_OK) st = check_output(y, y_dtype);
  if (st != CL_OK) return st;
  if ((st = check_work(work, work_bytes, cl_int8_work_bytes(tokens, N, K, 1))) != CL_OK) return st;
  launch_linear(product_of(codes, row, scale, tokens, w, w_row, w_scale, bias, N, K, y, y_row, work), K, y_dtype, static_cast<hipStream_t>(stream));
  return launched("int8 linear");
}

extern "C" cl_status cl_int8_forward(const void* x, int32_t dtype, int64_t x_row, int32_t tokens, float clamp,
                                     const int8_t* w, int64_t w_row, const float* w_scale, const float* bias, int32_t N,
                                     int32_t K, void* y, int32_t y_dtype, int64_t y_row, void* work, size_t work_bytes,
                                     void* stream) {
  clear_error();
  if (tokens < 0) return fail(CL_EINVAL, "int8: tokens must be >= 0");
  if (tokens == 0) return CL_OK;
  cl_status st = check_weights(w, w_row, w_scale, bias, N, K);
  if (st == CL_OK) st = check_values(x, dtype, K, clamp);
  if (st == CL_OK) st = check_output(y, y_dtype);
  if (st != CL_OK) return st;
  if ((st = check_work(work, work_bytes, cl_int8_work_bytes(tokens, N, K, 0))) != CL_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // sums, codes, scales
  int8_t* codes = static_cast<int8_t*>(work) + sums_bytes(tokens, N, K);
  float* scale = reinterpret_cast<float*>(codes + (size_t)tokens * padded(K));
  launch_quant(x, dtype, x_row, tokens, K, clamp, codes, padded(K), scale, s);
  launch_linear(product_of(codes, padded(K), scale, tokens, w, w_row, w_scale, bias, N, K, y, y_row, work), K, y_dtype, s);
  return launched("int8 forward");
}
