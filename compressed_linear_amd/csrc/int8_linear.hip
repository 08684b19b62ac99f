// int8_linear.hip -- the linear layer in 8-bit integers: rows of values to codes with a scale each, and the product
// of two sets of such rows.
#include <algorithm>

#include "cl_int8.h"
#include "serving.h"

namespace cl {
namespace {

constexpr int kMostK = 131071;  // 128 * 128 * K < 2^31
constexpr int kMostN = 1 << 25;
constexpr int64_t kMostRow = 1 << 23;  // 256 rows of it are within 32 bits
constexpr float kLeast = 0x1p-100f;

inline int64_t padded(int64_t K) { return (K + 127) / 128 * 128; }

// A value as it is quantised: clamped where there is a clamp (a NaN stays one).
__device__ __forceinline__ float clamped(float v, float clamp) { return clamp > 0.f && fabsf(v) > clamp ? copysignf(clamp, v) : v; }

// ------------------------------------------------------------------- codes
// A workgroup a row: its largest magnitude, as bits (a NaN is larger than any), then its codes.
template <int IN>
__global__ void __launch_bounds__(256) int8_quant_kernel(const typename Elem<IN>::raw* __restrict__ x, int64_t x_row, int64_t first, int K, int width,
                                                         float clamp, int8_t* __restrict__ codes, int64_t row, float* __restrict__ scale) {
  __shared__ uint32_t most[4];
  const int64_t t = first + blockIdx.x;
  x += t * x_row;
  uint32_t m = 0;
  for (int k = threadIdx.x; k < K; k += 256) m = max(m, __builtin_bit_cast(uint32_t, fabsf(clamped(Elem<IN>::up(x[k]), clamp))));
  for (int d = 32; d; d /= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(most[0], most[1]), max(most[2], most[3]));
  const float a = __builtin_bit_cast(float, m);
  const bool fine = m < 0x7f800000u, any = fine && a >= kLeast;
  const float s = any ? a * (1.f / 127.f) : fine ? 0.f : __builtin_nanf("");
  const float r = any ? 1.f / s : 0.f;
  if (threadIdx.x == 0) scale[t] = s;
  for (int k = threadIdx.x; k < width; k += 256)
    codes[t * row + k] = k < K && any ? (int8_t)fminf(fmaxf(rintf(clamped(Elem<IN>::up(x[k]), clamp) * r), -127.f), 127.f) : (int8_t)0;
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

__device__ __forceinline__ float scaled(const Product& p, int sum, float s, int n) {
  float v = (float)sum * s * p.w_scale[n];
  return p.bias ? v + p.bias[n] : v;
}

__device__ __forceinline__ void wait_loads() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
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
// directly, a step ahead, into the other of two buffers; a row's eight pieces of 16 bytes lie permuted by (row / 2) % 8, so that the 16
// lanes which LDS serves at once read all its banks.  A quarter step's operands are read between the products of the one before.  The
// one barrier of a step stands before its last quarter, whose operands are in registers: behind it the other buffer has arrived
// everywhere and this one is read by nobody.  Rows past the last give zeros (buffer loads with their bounds), and so do steps.
template <int OUT, int TW, int TT, int GW, int GT>
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
        __builtin_amdgcn_raw_ptr_buffer_load_lds(w, to, 16, at_row[i], step * 128, 0, 0);
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
  load(first, 0);
  wait_loads();
  meet();
  load(first + 1, 1);
  read(0, 0, 0);
  for (int at = first, buf = 0; at < end; ++at, buf ^= 1) {
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
    wait_loads();
    meet();
    load(at + 2, buf);
    read(buf ^ 1, 0, 0);
    multiply(1);
    mix(LOADS);
  }
  wait_lds();
  wait_loads();
  meet();
  // Out through LDS, 32 tokens of a wavefront at a time, so that rows are written in pieces of 16 bytes.
  typedef typename Result<OUT>::raw raw;
  constexpr int PITCH = FW * 32 * sizeof(raw) + 16, PER = 16 / sizeof(raw), ACROSS = FW * 32 / PER, DOWN = 64 / ACROSS;
  uint8_t* mine = lds + wave * (32 * PITCH);
  const int nb = n0 + ww * FW * 32;
  raw* y = OUT == kSums ? reinterpret_cast<raw*>(p.sums) + (int64_t)part * p.tokens * p.pitch : static_cast<raw*>(p.y);
  const int64_t y_row = OUT == kSums ? p.pitch : p.y_row;
  const bool whole = OUT == kSums || (reinterpret_cast<uintptr_t>(y) % 16 == 0 && y_row % PER == 0);
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
      const w4 v = *reinterpret_cast<const w4*>(mine + down * PITCH + across * sizeof(raw));
      if (t >= p.tokens || n >= p.N) continue;
      raw* out = y + t * y_row + n;
      if (whole && (OUT == kSums || n + PER <= p.N)) {
        *reinterpret_cast<w4*>(out) = v;
      } else {
#pragma unroll
        for (int e = 0; e < PER; ++e)
          if (n + e < p.N) {
            const uint32_t word = v[sizeof(raw) == 4 ? e : e / 2];
            if constexpr (sizeof(raw) == 4)
              out[e] = __builtin_bit_cast(raw, word);
            else
              out[e] = (raw)(word >> (16 * (e % 2)));
          }
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
// Two buffers of a step's rows, or 32 rows of each wavefront's outputs.
constexpr int lds_bytes(int tw, int tt, int waves, int out) {
  return 2 * (tw + tt) * 128 > waves * 32 * (out + 16) ? 2 * (tw + tt) * 128 : waves * 32 * (out + 16);
}
template <int OUT, int TW, int TT, int GW, int GT, bool HALVES>
__global__ void __launch_bounds__(64 * GW * GT, 2) int8_tile_kernel(Product p, Tiles g) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[lds_bytes(TW, TT, GW * GT, TW / GW * (int)sizeof(typename Result<OUT>::raw))];
  const bool half = HALVES && (int)blockIdx.x >= g.full;
  const int unit = half ? of_xcd(blockIdx.x - g.full, gridDim.x - g.full) : of_xcd(blockIdx.x, HALVES ? g.full : gridDim.x);
  const int tiles = g.t * g.w, at = half ? g.full + (unit >> 1) : unit, part = at / tiles, number = at % tiles;
  const int run = number / (8 * g.w), in = number % (8 * g.w), high = min(8, g.t - 8 * run);
  const int t0 = (8 * run + in % high) * TT, n0 = in / high * TW;
  const int first = (int)((int64_t)p.steps * part / g.parts), end = (int)((int64_t)p.steps * (part + 1) / g.parts);
  if constexpr (HALVES) {
    if (half) {
      const int t = t0 + (unit & 1) * (TT / 2);
      if (t < p.tokens) tile<OUT, TW, TT / 2, GW, GT>(p, lds, t, n0, first, end, part);
      return;
    }
  }
  tile<OUT, TW, TT, GW, GT>(p, lds, t0, n0, first, end, part);
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
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < p.N) y[e] = Elem<OUT>::down(scaled(p, sum[e], s, n + e));
}

// ------------------------------------------------------------- few tokens
// Up to 64 tokens: the weights are read once and nothing is shared but tokens, so operands come from memory into registers as they
// are (v_mfma_i32_16x16x64_i8; a lane has 32 bytes of a row in a step of 128 k, the same ones in both operands).  A workgroup has
// 16 FW outputs, its wavefronts take the steps in turn, and the sums meet in LDS.  AHEAD steps are asked for while as many are multiplied.
template <int OUT, int FW, int FT, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) int8_stream_kernel(Product p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int AHEAD = FW * FT >= 8 ? 1 : 2;
  __shared__ i4 sums[WAVES][FW][FT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = blockIdx.x * 16 * FW;
  const int r = lane & 15, at = lane >> 4;
  const int8_t* w_base = p.w + (int64_t)n0 * p.w_row;
  const uint32_t w_bytes = (uint32_t)(min(16 * FW, p.N - n0) * p.w_row), t_bytes = (uint32_t)(p.tokens * p.row);
  uint32_t w_at[FW], t_at[FT];
#pragma unroll
  for (int i = 0; i < FW; ++i) w_at[i] = (uint32_t)((16 * i + r) * p.w_row) + at * 32;
#pragma unroll
  for (int j = 0; j < FT; ++j) t_at[j] = (uint32_t)((16 * j + r) * p.row) + at * 32;
  i4 fw[2][AHEAD][FW][2], ft[2][AHEAD][FT][2];
  i4 acc[FW][FT] = {};
  const auto load = [&](int step, int to) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int k = step + a * WAVES;
      const auto w = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(w_base), 0, k < p.steps ? w_bytes : 0, 0x00020000);
      const auto t = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p.codes), 0, k < p.steps ? t_bytes : 0, 0x00020000);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < FW; ++i) fw[to][a][i][h] = __builtin_amdgcn_raw_buffer_load_b128(w, w_at[i] + 16 * h, k * 128, 2);
#pragma unroll
        for (int j = 0; j < FT; ++j) ft[to][a][j][h] = __builtin_amdgcn_raw_buffer_load_b128(t, t_at[j] + 16 * h, k * 128, 0);
      }
    }
  };
  const auto multiply = [&](int of) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < FW; ++i)
#pragma unroll
          for (int j = 0; j < FT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[of][a][i][h], ft[of][a][j][h], acc[i][j], 0, 0, 0);
  };
  load(wave, 0);
  for (int step = wave; step < p.steps; step += 2 * AHEAD * WAVES) {
    load(step + AHEAD * WAVES, 1);
    multiply(0);
    load(step + 2 * AHEAD * WAVES, 0);
    multiply(1);
  }
#pragma unroll
  for (int i = 0; i < FW; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) sums[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  // a lane of the sums has outputs 4 (l / 16) to + 3 of token l % 16
  for (int k = threadIdx.x; k < FW * FT * 64; k += 64 * WAVES) {
    const int l = k & 63, i = (k >> 6) % FW, j = (k >> 6) / FW, t = 16 * j + (l & 15), n = n0 + 16 * i + 4 * (l >> 4);
    i4 sum = sums[0][i][j][l];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += sums[w][i][j][l];
    if (t >= p.tokens) continue;
    const float s = p.scale[t];
    typename Elem<OUT>::raw* y = static_cast<typename Elem<OUT>::raw*>(p.y) + t * p.y_row + n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) y[e] = Elem<OUT>::down(scaled(p, sum[e], s, n + e));
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

template <int IN>
void launch_quant(const void* x, int64_t x_row, int rows, int K, float clamp, int8_t* codes, int64_t row, float* scale, hipStream_t s) {
  in_pieces(rows, 256, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL((int8_quant_kernel<IN>), dim3((unsigned)count), dim3(256), 0, s, static_cast<const typename Elem<IN>::raw*>(x), x_row, first,
                       K, (int)padded(K), clamp, codes, row, scale);
  });
}

void launch_quant(const void* x, int dtype, int64_t x_row, int rows, int K, float clamp, int8_t* codes, int64_t row, float* scale, hipStream_t s) {
  if (dtype == CL_F16)
    launch_quant<CL_F16>(x, x_row, rows, K, clamp, codes, row, scale, s);
  else if (dtype == CL_BF16)
    launch_quant<CL_BF16>(x, x_row, rows, K, clamp, codes, row, scale, s);
  else
    launch_quant<CL_F32>(x, x_row, rows, K, clamp, codes, row, scale, s);
}

// ------------------------------------------------------------------- plan
constexpr int kCus = 256;
constexpr int kFewTokens = 64;

// How a product is cut: the tile, parts of K.
struct Plan {
  int shape = 0, parts = 1;
};
struct Shape {
  int tw, tt;
  double step, twice;  // microseconds of a step of 128 k with one tile to each CU, and with two
};
constexpr Shape kShapes[] = {{256, 256, 1.85, 0}, {256, 192, 1.50, 0}, {256, 128, 1.05, 0}, {128, 128, 0.70, 1.10}};

int tiles_of(const Shape& s, int tokens, int N) { return ((tokens + s.tt - 1) / s.tt) * ((N + s.tw - 1) / s.tw); }

Plan plan_product(int tokens, int N, int K) {
  const int steps = (int)(padded(K) / 128);
  Plan best;
  if ((int64_t)tokens * N > (1 << 28)) return best;  // 4096 tiles: no parts, and the largest is the best
  double least = 1e30;
  for (int shape = 0; shape < 4; ++shape)
    for (int parts = 1; parts <= 16 && parts <= (steps + 7) / 8; ++parts) {
      const Shape& s = kShapes[shape];
      const int64_t n = (int64_t)tiles_of(s, tokens, N) * parts;
      const int64_t rounds = n / kCus, rest = n % kCus;
      double unit;  // in steps
      if (s.twice)
        unit = (n / (2 * kCus)) * s.twice + (n % (2 * kCus) > kCus ? s.twice : n % (2 * kCus) ? s.step : 0);
      else
        unit = rounds * s.step + (rest == 0 ? 0 : shape == 0 && parts == 1 && rest <= kCus / 2 ? kShapes[2].step : s.step);
      const double overhead = 6.0 * (double)((n + kCus - 1) / kCus);
      double t = unit * ((steps + parts - 1) / parts) + overhead;
      const double sums = 4.0 * tokens * N * parts;
      if (parts > 1) t += 4.0 + 2 * sums / 6e6;
      if (parts > 1 && sums > 268435456.0) continue;
      if (t < least) least = t, best = Plan{shape, parts};
    }
  return best;
}

size_t sums_bytes(int tokens, int N, int K) {
  if (tokens <= kFewTokens) return 0;
  const Plan p = plan_product(tokens, N, K);
  return p.parts > 1 ? (size_t)4 * p.parts * tokens * ((N + 3) / 4 * 4) : 0;
}

template <int OUT, int TW, int TT, int GW, int GT, bool HALVES>
void launch_tiles(const Product& p, int parts, hipStream_t s) {
  Tiles g{(p.tokens + TT - 1) / TT, (p.N + TW - 1) / TW, parts, 0};
  const int n = g.t * g.w * parts, rest = n % kCus;
  g.full = n;
  int blocks = n;
  if (HALVES && rest && rest <= kCus / 2) g.full = n - rest, blocks = g.full + 2 * rest;
  const auto kernel = int8_tile_kernel<OUT, TW, TT, GW, GT, HALVES>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * GW * GT), 0, s, p, g);
}

template <int OUT>
void launch_shape(const Product& p, const Plan& plan, hipStream_t s) {
  switch (plan.shape) {
    case 0: return launch_tiles<OUT, 256, 256, 4, 2, true>(p, plan.parts, s);
    case 1: return launch_tiles<OUT, 256, 192, 4, 2, false>(p, plan.parts, s);
    case 2: return launch_tiles<OUT, 256, 128, 4, 2, false>(p, plan.parts, s);
    default: return launch_tiles<OUT, 128, 128, 4, 2, false>(p, plan.parts, s);
  }
}

template <int OUT, int FW, int FT>
void launch_stream(const Product& p, hipStream_t s) {
  hipLaunchKernelGGL((int8_stream_kernel<OUT, FW, FT, 8>), dim3((unsigned)((p.N + 16 * FW - 1) / (16 * FW))), dim3(512), 0, s, p);
}

template <int OUT>
void launch_piece(const Product& p, int K, hipStream_t s) {
  if (p.tokens <= 16) return launch_stream<OUT, 1, 1>(p, s);
  if (p.tokens <= 32) return launch_stream<OUT, 2, 2>(p, s);
  if (p.tokens <= kFewTokens) return launch_stream<OUT, 2, 4>(p, s);
  const Plan plan = plan_product(p.tokens, p.N, K);
  if (plan.parts == 1) return launch_shape<OUT>(p, plan, s);
  launch_shape<kSums>(p, plan, s);
  in_pieces((int64_t)p.tokens * (p.pitch / 4), 1, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL((int8_join_kernel<OUT>), dim3((unsigned)((count + 255) / 256)), dim3(256), 0, s, p, plan.parts, first);
  });
}

// Tokens past what a launch holds (2^22 tiles of 512 threads) go in pieces.
template <int OUT>
void launch_linear(const Product& p, int K, hipStream_t s) {
  const int64_t most = std::max<int64_t>(1, (1 << 22) / ((p.N + 127) / 128) / 16) * 2048;
  for (int64_t first = 0; first < p.tokens; first += most) {
    Product q = p;
    q.codes += first * p.row;
    q.scale += first;
    q.y = beyond(p.y, OUT, first * p.y_row);
    q.tokens = (int)std::min(most, p.tokens - first);
    launch_piece<OUT>(q, K, s);
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
