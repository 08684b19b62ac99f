// rope_kv.hip -- rotary positions and the quantised K/V cache: its table,
// the rotation, appending tokens and reading them back.
#include <algorithm>
#include <type_traits>

#include "serving.h"

namespace cl {
namespace {

constexpr float kNan = __builtin_nanf("");

// ------------------------------------------------------------------- table
struct RopeScale {
  double base, inv_factor, lo, span, gain;  // base after NTK; YaRN ramp (i - lo) / span; gain m
  int yarn;
};

__global__ void __launch_bounds__(256) rope_table_kernel(float2* __restrict__ table, int positions, int half, int rot,
                                                         int64_t first, RopeScale r) {
  const int64_t at = first * half + (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= (int64_t)positions * half) return;
  const int p = (int)(at / half), i = (int)(at % half);
  double w = pow(r.base, -2.0 * i / rot);
  if (r.yarn) {
    const double ramp = fmin(fmax((i - r.lo) / r.span, 0.0), 1.0);
    w = w * r.inv_factor * ramp + w * (1.0 - ramp);
  } else {
    w = w * r.inv_factor;
  }
  double s, c;
  sincos(p * w, &s, &c);
  table[at] = make_float2((float)(c * r.gain), (float)(s * r.gain));
}

// ---------------------------------------------------------------- rotation
// The two channels of pair i.
__device__ __forceinline__ void pair_of(int layout, int half, int i, int* a, int* b) {
  *a = layout == CL_ROPE_HALF ? i : 2 * i;
  *b = layout == CL_ROPE_HALF ? i + half : 2 * i + 1;
}

// The axis of each pair, two bits to a pair, eight pairs to a half-word; positions are [axes, stride].  `used` has the bits of the
// axes that have pairs.
struct AxisMap {
  int64_t stride;
  int axes, used;
  uint32_t first[4];  // of[0] to of[7]
  uint16_t of[64];
};

struct RopeArgs {
  const void* x;
  void* y;
  const int32_t* positions;
  const float2* table;
  int64_t x_token, x_head, y_token, y_head;
  int tokens, heads, dim, rot, layout, table_rows;
};

// Arguments of a kernel for one axis or for several.  One axis does without the map, whose bytes every launch would carry (a call of
// cl_rope for one token 3.6 us instead of 3.0).
template <typename Args>
struct WithAxes : Args {
  AxisMap axes;
};
template <typename Args, bool AXES>
using ArgsOf = std::conditional_t<AXES, WithAxes<Args>, Args>;
static_assert(sizeof(ArgsOf<RopeArgs, false>) + sizeof(AxisMap) <= sizeof(ArgsOf<RopeArgs, true>), "one axis carries no map");

// The address of a token's position, where several axes have one each.
template <bool AXES, typename Args>
__device__ __forceinline__ const int32_t* position_at(const Args& a, int axis, int64_t t) {
  if constexpr (AXES)
    return a.positions + axis * a.axes.stride + t;
  else
    return a.positions + t;
}

// The axes of pairs 8u to 8u + 7.  Those of 64 pairs are in four words, which a lane picks from sooner than it reads them.
__device__ __forceinline__ uint32_t axes_of_8(const AxisMap& m, int u) {
  if (u >= 8) return m.of[u];
  const uint32_t a = u & 2 ? m.first[1] : m.first[0], b = u & 2 ? m.first[3] : m.first[2], w = u & 4 ? b : a;
  return (u & 1 ? w >> 16 : w) & 0xffff;
}
__device__ __forceinline__ int axis_of(const AxisMap& m, int pair) { return m.of[pair >> 3] >> (2 * (pair & 7)) & 3; }

// Any alignment: one thread a pair of channels, rotated or copied.
template <int IN, int OUT, bool AXES>
__global__ void __launch_bounds__(256) rope_pair_kernel(ArgsOf<RopeArgs, AXES> a) {
  const int pairs = (a.dim + 1) / 2, half = a.rot / 2;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= (int64_t)a.tokens * a.heads * pairs) return;
  const int i = (int)(at % pairs), h = (int)(at / pairs % a.heads), t = (int)(at / pairs / a.heads);
  const auto* x = static_cast<const typename Elem<IN>::raw*>(a.x) + t * a.x_token + h * a.x_head;
  auto* y = static_cast<typename Elem<OUT>::raw*>(a.y) + t * a.y_token + h * a.y_head;
  int c1, c2;
  if (i < half) {
    pair_of(a.layout, half, i, &c1, &c2);
  } else {
    c1 = 2 * i;
    c2 = 2 * i + 1 < a.dim ? 2 * i + 1 : c1;
  }
  float u = Elem<IN>::up(x[c1]), v = Elem<IN>::up(x[c2]);
  if (i < half) {
    int axis = 0;
    if constexpr (AXES) axis = axis_of(a.axes, i);
    const int p = *position_at<AXES>(a, axis, t);
    const bool in = p >= 0 && p < a.table_rows;
    const float2 cs = in ? a.table[(int64_t)p * half + i] : make_float2(kNan, kNan);
    rotate_pair(u, v, cs.x, cs.y);
  }
  y[c1] = Elem<OUT>::down(u);
  if (c2 != c1) y[c2] = Elem<OUT>::down(v);
}

// 16-byte pieces: a thread owns 16 channels of a head -- eight pairs, as two runs of 8 channels in either layout, or
// 16 channels that are copied -- of HEADS heads of a token, which then load its cosines and sines (from the caches for all
// heads but one) once.  Bound by memory, a step by the launch (72 heads of 128, fp32 to bf16: one token 2.4 us, 8192 tokens
// 81 us, 5.7 TB/s).  With several axes eight pairs of one axis are read as before, others pair by pair.
template <int IN, int OUT, int HEADS, bool AXES>
__global__ void __launch_bounds__(256) rope_kernel(ArgsOf<RopeArgs, AXES> a) {
  const int units = a.dim / 16, half = a.rot / 2, groups = (a.heads + HEADS - 1) / HEADS;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= (int64_t)a.tokens * groups * units) return;
  const int u = (int)(at % units), h = HEADS * (int)(at / units % groups), t = (int)(at / units / groups);
  const int n = min(HEADS, a.heads - h);
  const bool turned = 16 * u < a.rot;
  int c1 = 16 * u, c2 = c1 + 8;
  if (turned && a.layout == CL_ROPE_HALF) c1 = 8 * u, c2 = c1 + half;
  uint32_t of = 0;
  if constexpr (AXES) of = turned ? axes_of_8(a.axes, u) : 0;
  const bool one = of == (of & 3) * 0x5555;
  const int p = turned ? *position_at<AXES>(a, of & 3, t) : 0;
  const auto* x = static_cast<const typename Elem<IN>::raw*>(a.x) + t * a.x_token + h * a.x_head;
  auto* y = static_cast<typename Elem<OUT>::raw*>(a.y) + t * a.y_token + h * a.y_head;
  float v1[HEADS][8], v2[HEADS][8];
#pragma unroll
  for (int k = 0; k < HEADS; ++k) {
    if (k >= n) break;
    load8<IN>(x + k * a.x_head + c1, v1[k]);
    load8<IN>(x + k * a.x_head + c2, v2[k]);
  }
  if (turned) {
    float2 cs[8];
    if (!one) {
      if constexpr (AXES) {
        int on[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) on[k] = k < a.axes.axes ? *position_at<AXES>(a, k, t) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t axis = of >> (2 * i) & 3;
          const int q = axis & 2 ? (axis & 1 ? on[3] : on[2]) : (axis & 1 ? on[1] : on[0]);
          cs[i] = q >= 0 && q < a.table_rows ? a.table[(int64_t)q * half + 8 * u + i] : make_float2(kNan, kNan);
        }
      }
    } else if (p >= 0 && p < a.table_rows) {
      const float4* row = reinterpret_cast<const float4*>(a.table + (int64_t)p * half + 8 * u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = row[i];
        cs[2 * i] = make_float2(v.x, v.y), cs[2 * i + 1] = make_float2(v.z, v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = make_float2(kNan, kNan);
    }
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
      if (a.layout == CL_ROPE_HALF) {
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate_pair(v1[k][i], v2[k][i], cs[i].x, cs[i].y);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          rotate_pair(v1[k][2 * i], v1[k][2 * i + 1], cs[i].x, cs[i].y);
          rotate_pair(v2[k][2 * i], v2[k][2 * i + 1], cs[4 + i].x, cs[4 + i].y);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < HEADS; ++k) {
    if (k >= n) break;
    store8<OUT>(y + k * a.y_head + c1, v1[k]);
    store8<OUT>(y + k * a.y_head + c2, v2[k]);
  }
}

// Many tokens whose positions have several axes: a workgroup has a few tokens, gathers their cosines and sines into LDS, and then goes
// through their heads in the same pieces.
constexpr int kTurnPairs = 1024;
template <int IN, int OUT>
__global__ void __launch_bounds__(256) rope_axes_kernel(WithAxes<RopeArgs> a, int each) {
  __shared__ __attribute__((aligned(16))) float2 turn[kTurnPairs];
  const int units = a.dim / 16, half = a.rot / 2, first = blockIdx.x * each, tokens = min(each, a.tokens - first), pieces = a.heads * units;
  for (int i = threadIdx.x; i < tokens * half; i += 256) {
    const int k = i / half, pair = i % half;
    const int p = *position_at<true>(a, axis_of(a.axes, pair), first + k);
    turn[i] = p >= 0 && p < a.table_rows ? a.table[(int64_t)p * half + pair] : make_float2(kNan, kNan);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * pieces; i += 256) {
    const int k = i / pieces, at = i - k * pieces, h = at / units, u = at - h * units;
    const auto* x = static_cast<const typename Elem<IN>::raw*>(a.x) + (first + k) * a.x_token + h * a.x_head;
    auto* y = static_cast<typename Elem<OUT>::raw*>(a.y) + (first + k) * a.y_token + h * a.y_head;
    const bool turned = 16 * u < a.rot;
    int c1 = 16 * u, c2 = c1 + 8;
    if (turned && a.layout == CL_ROPE_HALF) c1 = 8 * u, c2 = c1 + half;
    float v1[8], v2[8];
    load8<IN>(x + c1, v1);
    load8<IN>(x + c2, v2);
    if (turned) {
      const float2* cs = turn + k * half + 8 * u;
      if (a.layout == CL_ROPE_HALF) {
#pragma unroll
        for (int j = 0; j < 8; ++j) rotate_pair(v1[j], v2[j], cs[j].x, cs[j].y);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          rotate_pair(v1[2 * j], v1[2 * j + 1], cs[j].x, cs[j].y);
          rotate_pair(v2[2 * j], v2[2 * j + 1], cs[4 + j].x, cs[4 + j].y);
        }
      }
    }
    store8<OUT>(y + c1, v1);
    store8<OUT>(y + c2, v2);
  }
}

// ------------------------------------------------------------------ append
struct AppendArgs {
  cl_kv_cache c;
  const void* src[2];  // k, v
  int64_t token[2], head[2];
  const int32_t* slots;
  const int32_t* positions;
  const float2* table;  // NULL: no rotation
  int tokens, rot, layout, table_rows, page_shift, side;
};

// Eight channels from `at` of a head at x; VEC: as two 16-byte (fp32) or one load, otherwise one by one.
template <int IN, bool VEC>
__device__ __forceinline__ void channels8(const typename Elem<IN>::raw* x, int at, float (&v)[8]) {
  if constexpr (VEC) {
    load8<IN>(x + at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<IN>::up(x[at + i]);
  }
}

// Largest value over the 16 lanes of a row (all get it), or over 8 or 4 of them.
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
  const auto step = [](float x, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v = fmaxf(v, step(v, std::integral_constant<int, 0xB1>()));                            // quad_perm [1, 0, 3, 2]
  v = fmaxf(v, step(v, std::integral_constant<int, 0x4E>()));                            // quad_perm [2, 3, 0, 1]
  if constexpr (LANES >= 8) v = fmaxf(v, step(v, std::integral_constant<int, 0x141>()));   // mirrored in 8
  if constexpr (LANES >= 16) v = fmaxf(v, step(v, std::integral_constant<int, 0x140>()));  // mirrored in 16
  return v;
}

// D / 8 lanes a (token, head, k or v), eight channels each; heads side by side in a workgroup as in the read, since the inputs are the
// larger part of the bytes and a token's heads lie together there (8192 tokens of 32 fp32 heads of 128, rotated, to int8: 71 us
// with 16 heads, 80 with 4, 83 with one).  Bound by memory for prompts, by the launch for steps.
template <int IN, int KIND, int D, bool VEC, bool AXES>
__global__ void __launch_bounds__(256) kv_append_kernel(ArgsOf<AppendArgs, AXES> a) {
  constexpr int LANES = D / 8;
  const int row_at = threadIdx.x / LANES, h = (blockIdx.y << a.side) + (row_at & ((1 << a.side) - 1)), which = blockIdx.z;
  const int tokens = 256 / LANES >> a.side, first = blockIdx.x * tokens, t = first + (row_at >> a.side);
  const int ch = 8 * (threadIdx.x % LANES);
  // With several axes a token's cosines and sines are gathered once for its heads in the workgroup.
  __shared__ float2 turn[AXES ? 256 / LANES : 1][D / 2];
  if constexpr (AXES) {
    if (which == 0) {
      const int half = a.rot / 2;
      for (int i = threadIdx.x; i < tokens * half; i += 256) {
        const int k = i / half, pair = i % half;
        if (first + k >= a.tokens) break;
        const int p = *position_at<true>(a, axis_of(a.axes, pair), first + k);
        turn[k][pair] = p >= 0 && p < a.table_rows ? a.table[(int64_t)p * half + pair] : make_float2(0.f, 0.f);
      }
      __syncthreads();
    }
  }
  if (t >= a.tokens) return;
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.c.pages << a.page_shift) return;
  const auto* x = static_cast<const typename Elem<IN>::raw*>(a.src[which]) + t * a.token[which] + h * a.head[which];
  float v[8];
  channels8<IN, VEC>(x, ch, v);
  if (a.table && which == 0) {
    const int half = a.rot / 2;
    const float2* cs;
    bool in = true;
    if constexpr (AXES) {
      cs = turn[row_at >> a.side];
      for (int k = 0; k < a.axes.axes; ++k) {
        const int p = *position_at<true>(a, k, t);
        in = in && (!(a.axes.used >> k & 1) || (p >= 0 && p < a.table_rows));
      }
    } else {
      const int p = a.positions[t];
      in = p >= 0 && p < a.table_rows;
      cs = a.table + (int64_t)(in ? p : 0) * half;
    }
    if (!in) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    } else if (VEC && a.layout == CL_ROPE_HALF) {  // half is a multiple of 8: the partners are 8 channels too
      if (ch < a.rot) {
        const bool low = ch < half;
        float w[8];
        channels8<IN, VEC>(x, low ? ch + half : ch - half, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 c = cs[(low ? ch : ch - half) + i];
          float p1 = low ? v[i] : w[i], p2 = low ? w[i] : v[i];
          rotate_pair(p1, p2, c.x, c.y);
          v[i] = low ? p1 : p2;
        }
      }
    } else if (VEC) {
      if (ch < a.rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = cs[ch / 2 + i];
          rotate_pair(v[2 * i], v[2 * i + 1], c.x, c.y);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (ch + i >= a.rot) continue;
        const int pr = a.layout == CL_ROPE_HALF ? (ch + i) % half : (ch + i) / 2;
        int c1, c2;
        pair_of(a.layout, half, pr, &c1, &c2);
        float p1 = Elem<IN>::up(x[c1]), p2 = Elem<IN>::up(x[c2]);
        const float2 c = cs[pr];
        rotate_pair(p1, p2, c.x, c.y);
        v[i] = ch + i == c1 ? p1 : p2;
      }
    }
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = v[i] == v[i] ? v[i] : 0.f;  // a NaN counts as 0
    m = fmaxf(m, fabsf(v[i]));
  }
  m = lanes_max<KIND == CL_KV_INT8 ? LANES : 4>(m);  // a scale's lanes: a head, or 32 channels
  constexpr float most = KIND == CL_KV_INT8 ? 127.f : 7.f;
  float s = fminf(m / most, KIND == CL_KV_INT8 ? 65504.f : 8192.f);
  if (KIND == CL_KV_INT4) s = (float)(__bf16)s;
  const _Float16 s16 = (_Float16)s;
  const float r = (float)s16 > 0.f ? 1.0f / (float)s16 : 0.f;
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // an infinity times 0 would be NaN, but then the scale is not 0
    const float c = fminf(fmaxf(rintf(v[i] * r), -most), most);
    q[i] = (uint32_t)(int)(c + (KIND == CL_KV_INT8 ? 128.f : 8.f));
  }
  const int64_t row = (((int64_t)(slot >> a.page_shift) * a.c.heads + h) << a.page_shift) + (slot & (a.c.page_size - 1));
  uint8_t* out = static_cast<uint8_t*>(which ? a.c.v : a.c.k);
  uint16_t* sc = which ? a.c.v_scale : a.c.k_scale;
  if (KIND == CL_KV_INT8) {
    *reinterpret_cast<w2*>(out + row * D + ch) =
        w2{q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24, q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24};
    if (ch == 0) sc[row] = __builtin_bit_cast(uint16_t, s16);
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= q[i] << (4 * i);
    *reinterpret_cast<uint32_t*>(out + row * (D / 2) + ch / 2) = w;
    if (ch % 32 == 0) sc[row * (D / 32) + ch / 32] = __builtin_bit_cast(uint16_t, s16);
  }
}

// -------------------------------------------------------------------- read
// D / 8 lanes a (slot, head), eight channels of K and of V each, two slots to a thread.  A workgroup has `1 << side` heads
// side by side, the largest power of two up to 16 that divides the heads: the outputs are the larger part of the bytes, and a
// slot's heads lie together there (32 heads of 128, 40000 slots: 200 us with 16 heads, 215 with 4, 228 with one).
// Bound by memory.
template <int OUT, int KIND, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(cl_kv_cache c, int page_shift, int side, const int32_t* __restrict__ slots, int n,
                                                      typename Elem<OUT>::raw* __restrict__ ko,
                                                      typename Elem<OUT>::raw* __restrict__ vo) {
  constexpr int LANES = D / 8, ROWS = 256 / LANES, PER = 2;
  const int r = threadIdx.x / LANES, h = (blockIdx.y << side) + (r & ((1 << side) - 1)), ch = 8 * (threadIdx.x % LANES);
  const int apart = ROWS >> side, t0 = blockIdx.x * (apart * PER) + (r >> side);
  w2 code[PER][2];
  float scale[PER][2];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int t = t0 + k * apart;
    const int slot = t < n ? slots[t] : -1;
    const bool in = slot >= 0 && slot < c.pages << page_shift;
    const int64_t row = in ? (((int64_t)(slot >> page_shift) * c.heads + h) << page_shift) + (slot & (c.page_size - 1)) : 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint8_t* b = static_cast<const uint8_t*>(w ? c.v : c.k);
      const uint16_t* s = w ? c.v_scale : c.k_scale;
      if constexpr (KIND == CL_KV_INT8) {
        code[k][w] = *reinterpret_cast<const w2*>(b + row * D + ch);
        scale[k][w] = Elem<CL_F16>::up(s[row]);
      } else {
        code[k][w].x = *reinterpret_cast<const uint32_t*>(b + row * (D / 2) + ch / 2);
        scale[k][w] = Elem<CL_F16>::up(s[row * (D / 32) + ch / 32]);
      }
      if (!in) scale[k][w] = 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int t = t0 + k * apart;
    if (t >= n) break;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = KIND == CL_KV_INT8 ? (int)((code[k][w][i / 4] >> (8 * (i % 4))) & 255) - 128
                                         : (int)((code[k][w].x >> (4 * i)) & 15) - 8;
        v[i] = (float)q * scale[k][w];
      }
      store8<OUT>((w ? vo : ko) + ((int64_t)t * c.heads + h) * D + ch, v);
    }
  }
}

// The largest power of two (its logarithm) up to 16 that divides the heads.
int heads_side_by_side(int heads) { return std::min(__builtin_ctz(heads), 4); }

// A launch's part of a call: tokens [first, first + count).
template <typename Args>
Args piece_of(Args a, int in, int out, int64_t first, int64_t count) {
  a.x = beyond(a.x, in, first * a.x_token);
  a.y = beyond(a.y, out, first * a.y_token);
  a.positions += first;
  a.tokens = (int)count;
  return a;
}

template <int IN, int OUT>
void launch_rope(const WithAxes<RopeArgs>& a, hipStream_t s) {
  const bool vec = a.rot % 16 == 0 && a.dim % 16 == 0 && aligned_to(a.table, 16) &&
                   heads_aligned(a.x, IN, a.x_token, a.x_head) && heads_aligned(a.y, OUT, a.y_token, a.y_head);
  const auto go = [&](auto kernel, const auto& args, int64_t each) {
    in_pieces(a.tokens, each, [&](int64_t first, int64_t count) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)((count * each + 255) / 256)), dim3(256), 0, s, piece_of(args, IN, OUT, first, count));
    });
  };
  const RopeArgs& plain = a;
  if (a.axes.axes > 1) {
    const bool many = (int64_t)a.tokens * a.heads >= (1 << 14), wide = IN == CL_F32 && (int64_t)a.tokens * a.heads >= (1 << 17);
    if (!vec) {
      go(rope_pair_kernel<IN, OUT, true>, a, (int64_t)a.heads * ((a.dim + 1) / 2));
    } else if (many && !wide) {
      // 8192 x 72 heads of 128, bf16, axes in turns: 56.8 us (one axis 54); by the kernel of few tokens 73.5, with two or four tokens to a
      // workgroup 60.7 and 64.5.  Wide fp32 heads cover the gathering: to bf16 83.2 us by the kernel of few tokens, 85.3 here; to fp32 118
      // and 114.
      const int each = std::max(1, std::min(kTurnPairs / (a.rot / 2), 512 / (a.heads * (a.dim / 16))));
      in_pieces(a.tokens, 256, [&](int64_t first, int64_t count) {
        hipLaunchKernelGGL((rope_axes_kernel<IN, OUT>), dim3((unsigned)((count + each - 1) / each)), dim3(256), 0, s,
                           piece_of(a, IN, OUT, first, count), each);
      });
    } else {
      go(rope_kernel<IN, OUT, 1, true>, a, (int64_t)a.heads * (a.dim / 16));
    }
    return;
  }
  if (!vec)
    go(rope_pair_kernel<IN, OUT, false>, plain, (int64_t)a.heads * ((a.dim + 1) / 2));
  // Two heads to a thread for many tokens of 16 bits, whose heads are no larger than the cosines and sines (8192 x 72 heads, half
  // of each rotated: 53 us, 55.5 with one and 54 with four; fp32 83 against 81.5; 64 tokens 3.3 against 3.0).
  else if (IN != CL_F32 && (int64_t)a.tokens * a.heads >= (1 << 17))
    go(rope_kernel<IN, OUT, 2, false>, plain, (int64_t)((a.heads + 1) / 2) * (a.dim / 16));
  else
    go(rope_kernel<IN, OUT, 1, false>, plain, (int64_t)a.heads * (a.dim / 16));
}

template <int IN>
void launch_rope(int out, const WithAxes<RopeArgs>& a, hipStream_t s) {
  if (out == CL_F16)
    launch_rope<IN, CL_F16>(a, s);
  else if (out == CL_BF16)
    launch_rope<IN, CL_BF16>(a, s);
  else
    launch_rope<IN, CL_F32>(a, s);
}

template <int IN, int KIND, int D, bool AXES>
void launch_append(const ArgsOf<AppendArgs, AXES>& a, hipStream_t s) {
  const bool vec = heads_aligned(a.src[0], IN, a.token[0], a.head[0]) && heads_aligned(a.src[1], IN, a.token[1], a.head[1]) &&
                   a.rot % 16 == 0;
  const int each = 256 / (D / 8) >> a.side;  // tokens of a workgroup
  in_pieces(a.tokens, (D / 8) << a.side, [&](int64_t first, int64_t count) {
    auto b = a;
    for (int w = 0; w < 2; ++w) b.src[w] = beyond(a.src[w], IN, first * a.token[w]);
    b.slots += first;
    if (a.table) b.positions += first;
    b.tokens = (int)count;
    const dim3 grid((unsigned)((count + each - 1) / each), a.c.heads >> a.side, 2);
    const auto kernel = vec ? kv_append_kernel<IN, KIND, D, true, AXES> : kv_append_kernel<IN, KIND, D, false, AXES>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, b);
  });
}

template <int IN, int KIND, int D>
void launch_append(const WithAxes<AppendArgs>& a, hipStream_t s) {
  if (a.table && a.axes.axes > 1)
    launch_append<IN, KIND, D, true>(a, s);
  else
    launch_append<IN, KIND, D, false>(a, s);
}

template <int IN>
void launch_append(const WithAxes<AppendArgs>& a, hipStream_t s) {
  if (a.c.kind == CL_KV_INT8) {
    if (a.c.dim == 128)
      launch_append<IN, CL_KV_INT8, 128>(a, s);
    else
      launch_append<IN, CL_KV_INT8, 64>(a, s);
  } else {
    if (a.c.dim == 128)
      launch_append<IN, CL_KV_INT4, 128>(a, s);
    else
      launch_append<IN, CL_KV_INT4, 64>(a, s);
  }
}

template <int OUT, int KIND, int D>
void launch_read(const cl_kv_cache& c, const int32_t* slots, int n, void* ko, void* vo, hipStream_t s) {
  typedef typename Elem<OUT>::raw raw;
  const int side = heads_side_by_side(c.heads), slots_each = 2 * 256 / (D / 8) >> side;
  in_pieces(n, (D / 8) << side, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL((kv_read_kernel<OUT, KIND, D>), dim3((unsigned)((count + slots_each - 1) / slots_each), c.heads >> side),
                       dim3(256), 0, s, c, __builtin_ctz(c.page_size), side, slots + first, (int)count,
                       static_cast<raw*>(ko) + first * c.heads * D, static_cast<raw*>(vo) + first * c.heads * D);
  });
}

template <int OUT>
void launch_read(const cl_kv_cache& c, const int32_t* slots, int n, void* ko, void* vo, hipStream_t s) {
  if (c.kind == CL_KV_INT8) {
    if (c.dim == 128)
      launch_read<OUT, CL_KV_INT8, 128>(c, slots, n, ko, vo, s);
    else
      launch_read<OUT, CL_KV_INT8, 64>(c, slots, n, ko, vo, s);
  } else {
    if (c.dim == 128)
      launch_read<OUT, CL_KV_INT4, 128>(c, slots, n, ko, vo, s);
    else
      launch_read<OUT, CL_KV_INT4, 64>(c, slots, n, ko, vo, s);
  }
}

}  // namespace
}  // namespace cl

using namespace cl;

extern "C" cl_status cl_rope_table(int32_t positions, int32_t rot, double base, int32_t scaling, double factor,
                                   int32_t trained, double beta_fast, double beta_slow, float* table, void* stream) {
  clear_error();
  if (positions < 1 || rot < 2 || rot % 2) return fail(CL_EINVAL, "rope table: positions >= 1 and an even rot >= 2 are wanted");
  if (rot > 1024) return fail(CL_ESIZE, "rope table: rot %d above 1024", rot);
  if (!table || !aligned_to(table, 8)) return fail(CL_EINVAL, "rope table: table is NULL or not 8-byte aligned");
  if (!(base > 1.0) || !(base < 1e300)) return fail(CL_EINVAL, "rope table: base must be finite and above 1");
  if (scaling < CL_ROPE_NONE || scaling > CL_ROPE_YARN) return fail(CL_EINVAL, "rope table: unknown scaling %d", scaling);
  if (scaling != CL_ROPE_NONE && (!(factor >= 1.0) || !(factor < 1e6)))
    return fail(CL_EINVAL, "rope table: factor must be in [1, 1e6)");
  RopeScale r = {base, 1.0, 0.0, 1.0, 1.0, 0};
  if (scaling == CL_ROPE_LINEAR) r.inv_factor = 1.0 / factor;
  if (scaling == CL_ROPE_NTK) {
    if (rot < 4) return fail(CL_EINVAL, "rope table: NTK needs rot >= 4");
    r.base = base * pow(factor, (double)rot / (rot - 2));
  }
  if (scaling == CL_ROPE_YARN) {
    if (trained < 1 || !(beta_slow > 0) || !(beta_fast > beta_slow) || !(beta_fast < 1e9))
      return fail(CL_EINVAL, "rope table: YARN needs trained >= 1 and beta_fast > beta_slow > 0");
    const double two_pi = 6.283185307179586;
    double lo = floor(rot * log(trained / (beta_fast * two_pi)) / (2 * log(base)));
    double hi = ceil(rot * log(trained / (beta_slow * two_pi)) / (2 * log(base)));
    lo = lo < 0 ? 0 : lo > rot - 1 ? rot - 1 : lo;
    hi = hi < 0 ? 0 : hi > rot - 1 ? rot - 1 : hi;
    r.yarn = 1;
    r.inv_factor = 1.0 / factor;
    r.lo = lo;
    r.span = hi - lo > 0.001 ? hi - lo : 0.001;
    r.gain = 0.1 * log(factor) + 1.0;
  }
  in_pieces(positions, rot / 2, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)((count * (rot / 2) + 255) / 256)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), reinterpret_cast<float2*>(table), (int)(first + count), rot / 2, rot, first, r);
  });
  return launched("rope table");
}

namespace {

// The axis of every pair of a rotation over `rot` channels; no sections: one axis.
cl_status axis_map(const int32_t* sections, int axes, int order, int rot, int tokens, AxisMap* m) {
  m->axes = 1;
  if (!sections) return CL_OK;  // nothing else is read
  *m = AxisMap{tokens, 1, 1, {}, {}};
  if (axes < 1 || axes > 4) return fail(CL_EINVAL, "rope: %d axes (1 to 4 are wanted)", axes);
  if (order != CL_ROPE_BLOCKS && order != CL_ROPE_TURNS) return fail(CL_EINVAL, "rope: unknown order %d of the axes", order);
  const int half = rot / 2;
  int64_t sum = 0;
  for (int k = 0; k < axes; ++k) {
    if (sections[k] < 0) return fail(CL_EINVAL, "rope: a section of %d pairs", sections[k]);
    sum += sections[k];
    if (order == CL_ROPE_TURNS && k && sections[k] && k + (int64_t)axes * (sections[k] - 1) >= half)
      return fail(CL_EINVAL, "rope: axis %d does not get %d turns among %d pairs", k, sections[k], half);
  }
  if (sum != half) return fail(CL_EINVAL, "rope: sections of %lld pairs, the table has %d", (long long)sum, half);
  m->axes = axes;
  m->used = 0;
  for (int i = 0, k = 0, end = sections[0]; i < half; ++i) {
    int axis = i % axes;
    if (order == CL_ROPE_BLOCKS) {
      while (i >= end) end += sections[++k];
      axis = k;
    } else if (i / axes >= sections[axis]) {
      axis = 0;
    }
    m->of[i / 8] |= (uint16_t)(axis << (2 * (i % 8)));
    m->used |= 1 << axis;
  }
  for (int u = 0; u < 8; ++u) m->first[u / 2] |= (uint32_t)m->of[u] << (16 * (u % 2));
  return CL_OK;
}

}  // namespace

extern "C" cl_status cl_rope(const void* x, int32_t x_dtype, int64_t x_token, int64_t x_head, int32_t tokens,
                             int32_t heads, int32_t dim, const int32_t* positions, const float* table,
                             int32_t table_rows, int32_t rot, int32_t layout, void* y, int32_t y_dtype, int64_t y_token,
                             int64_t y_head, void* stream) {
  return cl_rope_axes(x, x_dtype, x_token, x_head, tokens, heads, dim, positions, 1, nullptr, CL_ROPE_BLOCKS, table, table_rows,
                      rot, layout, y, y_dtype, y_token, y_head, stream);
}

extern "C" cl_status cl_rope_axes(const void* x, int32_t x_dtype, int64_t x_token, int64_t x_head, int32_t tokens,
                                  int32_t heads, int32_t dim, const int32_t* positions, int32_t axes,
                                  const int32_t* sections, int32_t order, const float* table, int32_t table_rows,
                                  int32_t rot, int32_t layout, void* y, int32_t y_dtype, int64_t y_token, int64_t y_head,
                                  void* stream) {
  clear_error();
  if (tokens < 0 || heads < 1 || dim < 2) return fail(CL_EINVAL, "rope: tokens >= 0, heads >= 1 and dim >= 2 are wanted");
  if (!elem_ok(x_dtype) || !elem_ok(y_dtype)) return fail(CL_EINVAL, "rope: unknown element type");
  if (dim > 1024) return fail(CL_ESIZE, "rope: dim %d above 1024", dim);
  if (tokens == 0) return CL_OK;
  if (!x || !y) return fail(CL_EINVAL, "rope: x or y is NULL");
  if (!aligned_to(x, elem_size(x_dtype)) || !aligned_to(y, elem_size(y_dtype)))
    return fail(CL_EINVAL, "rope: x or y is misaligned for its type");
  cl_status st = check_rope(positions, table, table_rows, rot, layout, dim);
  if (st != CL_OK) return st;
  if (y == x && (x_dtype != y_dtype || x_token != y_token || x_head != y_head))
    return fail(CL_EINVAL, "rope: y may be x only with the same type and strides");
  if ((int64_t)tokens * heads >= ((int64_t)1 << 40) / dim) return fail(CL_ESIZE, "rope: tokens * heads * dim at 2^40 or more");
  WithAxes<RopeArgs> a;
  static_cast<RopeArgs&>(a) = {x, y, positions, reinterpret_cast<const float2*>(table), x_token, x_head, y_token, y_head,
                               tokens, heads, dim, rot, layout, table_rows};
  if ((st = axis_map(sections, axes, order, rot, tokens, &a.axes)) != CL_OK) return st;
  if ((int64_t)heads * ((dim + 1) / 2) > kLaunch) return fail(CL_ESIZE, "rope: too many heads");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (x_dtype == CL_F16)
    launch_rope<CL_F16>(y_dtype, a, s);
  else if (x_dtype == CL_BF16)
    launch_rope<CL_BF16>(y_dtype, a, s);
  else
    launch_rope<CL_F32>(y_dtype, a, s);
  return launched("rope");
}

extern "C" cl_status cl_kv_append(const cl_kv_cache* cache, const void* k, const void* v, int32_t dtype, int32_t tokens,
                                  int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                                  const int32_t* slots, const int32_t* positions, const float* table,
                                  int32_t table_rows, int32_t rot, int32_t layout, void* stream) {
  return cl_kv_append_axes(cache, k, v, dtype, tokens, k_token, k_head, v_token, v_head, slots, positions, 1, nullptr,
                           CL_ROPE_BLOCKS, table, table_rows, rot, layout, stream);
}

extern "C" cl_status cl_kv_append_axes(const cl_kv_cache* cache, const void* k, const void* v, int32_t dtype,
                                       int32_t tokens, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                                       const int32_t* slots, const int32_t* positions, int32_t axes,
                                       const int32_t* sections, int32_t order, const float* table, int32_t table_rows,
                                       int32_t rot, int32_t layout, void* stream) {
  clear_error();
  cl_status st = check_cache(cache);
  if (st != CL_OK) return st;
  if (tokens < 0) return fail(CL_EINVAL, "append: tokens must be >= 0");
  if (!elem_ok(dtype)) return fail(CL_EINVAL, "append: unknown element type");
  if (tokens == 0) return CL_OK;
  if (!k || !v || !slots) return fail(CL_EINVAL, "append: a required pointer is NULL");
  if (!aligned_to(k, elem_size(dtype)) || !aligned_to(v, elem_size(dtype)) || !aligned_to(slots, 4))
    return fail(CL_EINVAL, "append: a pointer is misaligned for its type");
  if (table && (st = check_rope(positions, table, table_rows, rot, layout, cache->dim)) != CL_OK) return st;
  WithAxes<AppendArgs> a;
  static_cast<AppendArgs&>(a) = {*cache, {k, v}, {k_token, v_token}, {k_head, v_head}, slots, positions, reinterpret_cast<const float2*>(table),
                                 tokens, table ? rot : 0, layout, table_rows, __builtin_ctz(cache->page_size), heads_side_by_side(cache->heads)};
  if (table && (st = axis_map(sections, axes, order, rot, tokens, &a.axes)) != CL_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == CL_F16)
    launch_append<CL_F16>(a, s);
  else if (dtype == CL_BF16)
    launch_append<CL_BF16>(a, s);
  else
    launch_append<CL_F32>(a, s);
  return launched("append");
}

extern "C" cl_status cl_kv_read(const cl_kv_cache* cache, const int32_t* slots, int32_t n, void* k_out, void* v_out,
                                int32_t dtype, void* stream) {
  clear_error();
  cl_status st = check_cache(cache);
  if (st != CL_OK) return st;
  if (n < 0) return fail(CL_EINVAL, "read: n must be >= 0");
  if (!elem_ok(dtype)) return fail(CL_EINVAL, "read: unknown element type");
  if (n == 0) return CL_OK;
  if (!slots || !k_out || !v_out) return fail(CL_EINVAL, "read: a required pointer is NULL");
  if (!aligned_to(k_out, 16) || !aligned_to(v_out, 16) || !aligned_to(slots, 4))
    return fail(CL_EINVAL, "read: outputs must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == CL_F16)
    launch_read<CL_F16>(*cache, slots, n, k_out, v_out, s);
  else if (dtype == CL_BF16)
    launch_read<CL_BF16>(*cache, slots, n, k_out, v_out, s);
  else
    launch_read<CL_F32>(*cache, slots, n, k_out, v_out, s);
  return launched("read");
}
