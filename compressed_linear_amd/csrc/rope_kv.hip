// rope_kv.hip -- rotary positions and the quantised K/V cache: its table,
// the rotation, appending tokens and reading them back.
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
                                                         RopeScale r) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
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

struct RopeArgs {
  const void* x;
  void* y;
  const int32_t* positions;
  const float2* table;
  int64_t x_token, x_head, y_token, y_head;
  int tokens, heads, dim, rot, layout, table_rows;
};

// One thread a pair of channels, rotated or copied.
template <int IN, int OUT>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a) {
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
    const int p = a.positions[t];
    const bool in = p >= 0 && p < a.table_rows;
    const float2 cs = in ? a.table[(int64_t)p * half + i] : make_float2(kNan, kNan);
    rotate_pair(u, v, cs.x, cs.y);
  }
  y[c1] = Elem<OUT>::down(u);
  if (c2 != c1) y[c2] = Elem<OUT>::down(v);
}

// ------------------------------------------------------------------ append
struct AppendArgs {
  cl_kv_cache c;
  const void* src[2];  // k, v
  int64_t token[2], head[2];
  const int32_t* slots;
  const int32_t* positions;
  const float2* table;  // NULL: no rotation
  int tokens, rot, layout, table_rows;
};

__device__ __forceinline__ int64_t cache_row(const cl_kv_cache& c, int slot, int head) {
  const int page = slot / c.page_size;
  return ((int64_t)page * c.heads + head) * c.page_size + slot % c.page_size;
}

// One wavefront a (token, head, k or v); lane l holds channels 2l and 2l + 1.
template <int IN, int KIND>
__global__ void __launch_bounds__(64) kv_append_kernel(AppendArgs a) {
  const int t = blockIdx.x, h = blockIdx.y, which = blockIdx.z, l = threadIdx.x;
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.c.pages * a.c.page_size) return;
  const int D = a.c.dim, half = a.rot / 2;
  const auto* x = static_cast<const typename Elem<IN>::raw*>(a.src[which]) + t * a.token[which] + h * a.head[which];
  float v[2] = {0.f, 0.f};
  const bool rotated = a.table && which == 0;
  const int p = rotated ? a.positions[t] : 0;
  const bool in = !rotated || (p >= 0 && p < a.table_rows);
  for (int j = 0; j < 2; ++j) {
    const int ch = 2 * l + j;
    if (ch >= D || !in) continue;
    float own = Elem<IN>::up(x[ch]);
    if (rotated && ch < a.rot) {
      const int i = a.layout == CL_ROPE_HALF ? ch % half : ch / 2;
      int c1, c2;
      pair_of(a.layout, half, i, &c1, &c2);
      float u = Elem<IN>::up(x[c1]), w = Elem<IN>::up(x[c2]);
      const float2 cs = a.table[(int64_t)p * half + i];
      rotate_pair(u, w, cs.x, cs.y);
      own = ch == c1 ? u : w;
    }
    v[j] = own == own ? own : 0.f;
  }
  float m = fmaxf(fabsf(v[0]), fabsf(v[1]));
  const int width = KIND == CL_KV_INT8 ? 64 : 16;  // lanes of a scale: a head, or 32 channels
  for (int d = 1; d < width; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const int64_t row = cache_row(a.c, slot, h);
  uint8_t* out = static_cast<uint8_t*>(which ? a.c.v : a.c.k);
  uint16_t* sc = which ? a.c.v_scale : a.c.k_scale;
  const int most = KIND == CL_KV_INT8 ? 127 : 7;
  float s = fminf(m / (float)most, KIND == CL_KV_INT8 ? 65504.f : 8192.f);
  if (KIND == CL_KV_INT4) s = (float)(__bf16)s;
  const _Float16 s16 = (_Float16)s;
  const float r = (float)s16 > 0.f ? 1.0f / (float)s16 : 0.f;
  int q[2];
  for (int j = 0; j < 2; ++j) {
    const float c = r > 0.f ? rintf(v[j] * r) : 0.f;
    q[j] = (int)fminf(fmaxf(c, (float)-most), (float)most);
  }
  if (2 * l >= D) return;
  if (KIND == CL_KV_INT8) {
    out[row * D + 2 * l] = (uint8_t)(q[0] + 128);
    out[row * D + 2 * l + 1] = (uint8_t)(q[1] + 128);
    if (l == 0) sc[row] = __builtin_bit_cast(uint16_t, s16);
  } else {
    out[row * (D / 2) + l] = (uint8_t)((q[0] + 8) | (q[1] + 8) << 4);
    if (l % 16 == 0) sc[row * (D / 32) + l / 16] = __builtin_bit_cast(uint16_t, s16);
  }
}

// -------------------------------------------------------------------- read
// One thread a channel of K and of V.
template <int OUT, int KIND>
__global__ void __launch_bounds__(256) kv_read_kernel(cl_kv_cache c, const int32_t* __restrict__ slots, int n,
                                                      typename Elem<OUT>::raw* __restrict__ ko,
                                                      typename Elem<OUT>::raw* __restrict__ vo) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int D = c.dim;
  if (at >= (int64_t)n * c.heads * D) return;
  const int ch = (int)(at % D), h = (int)(at / D % c.heads), t = (int)(at / D / c.heads);
  const int slot = slots[t];
  float v[2] = {0.f, 0.f};
  if (slot >= 0 && slot < c.pages * c.page_size) {
    const int64_t row = cache_row(c, slot, h);
    for (int w = 0; w < 2; ++w) {
      const uint8_t* b = static_cast<const uint8_t*>(w ? c.v : c.k);
      const uint16_t* s = w ? c.v_scale : c.k_scale;
      if (KIND == CL_KV_INT8) {
        v[w] = (float)((int)b[row * D + ch] - 128) * Elem<CL_F16>::up(s[row]);
      } else {
        const int nib = (b[row * (D / 2) + ch / 2] >> (ch % 2 * 4)) & 15;
        v[w] = (float)(nib - 8) * Elem<CL_F16>::up(s[row * (D / 32) + ch / 32]);
      }
    }
  }
  ko[at] = Elem<OUT>::down(v[0]);
  vo[at] = Elem<OUT>::down(v[1]);
}

template <int IN>
void launch_rope(int out, const RopeArgs& a, unsigned grid, hipStream_t s) {
  if (out == CL_F16)
    hipLaunchKernelGGL((rope_kernel<IN, CL_F16>), dim3(grid), dim3(256), 0, s, a);
  else if (out == CL_BF16)
    hipLaunchKernelGGL((rope_kernel<IN, CL_BF16>), dim3(grid), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((rope_kernel<IN, CL_F32>), dim3(grid), dim3(256), 0, s, a);
}

template <int IN>
void launch_append(const AppendArgs& a, hipStream_t s) {
  const dim3 grid(a.tokens, a.c.heads, 2);
  if (a.c.kind == CL_KV_INT8)
    hipLaunchKernelGGL((kv_append_kernel<IN, CL_KV_INT8>), grid, dim3(64), 0, s, a);
  else
    hipLaunchKernelGGL((kv_append_kernel<IN, CL_KV_INT4>), grid, dim3(64), 0, s, a);
}

template <int OUT>
void launch_read(const cl_kv_cache& c, const int32_t* slots, int n, void* ko, void* vo, unsigned grid, hipStream_t s) {
  typedef typename Elem<OUT>::raw raw;
  if (c.kind == CL_KV_INT8)
    hipLaunchKernelGGL((kv_read_kernel<OUT, CL_KV_INT8>), dim3(grid), dim3(256), 0, s, c, slots, n,
                       static_cast<raw*>(ko), static_cast<raw*>(vo));
  else
    hipLaunchKernelGGL((kv_read_kernel<OUT, CL_KV_INT4>), dim3(grid), dim3(256), 0, s, c, slots, n,
                       static_cast<raw*>(ko), static_cast<raw*>(vo));
}

// Workgroups of 256 threads for n threads; 0 where the grid would be too large.
unsigned grid_of(int64_t n) {
  const int64_t g = (n + 255) / 256;
  return g > 0x7FFFFFFFll ? 0u : (unsigned)g;
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
  const unsigned grid = grid_of((int64_t)positions * (rot / 2));
  if (!grid) return fail(CL_ESIZE, "rope table: too many positions");
  hipLaunchKernelGGL(rope_table_kernel, dim3(grid), dim3(256), 0, static_cast<hipStream_t>(stream),
                     reinterpret_cast<float2*>(table), positions, rot / 2, rot, r);
  return launched("rope table");
}

extern "C" cl_status cl_rope(const void* x, int32_t x_dtype, int64_t x_token, int64_t x_head, int32_t tokens,
                             int32_t heads, int32_t dim, const int32_t* positions, const float* table,
                             int32_t table_rows, int32_t rot, int32_t layout, void* y, int32_t y_dtype, int64_t y_token,
                             int64_t y_head, void* stream) {
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
  const RopeArgs a = {x, y, positions, reinterpret_cast<const float2*>(table), x_token, x_head, y_token, y_head,
                      tokens, heads, dim, rot, layout, table_rows};
  const unsigned grid = grid_of((int64_t)tokens * heads * ((dim + 1) / 2));
  if (!grid) return fail(CL_ESIZE, "rope: too many tokens");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (x_dtype == CL_F16)
    launch_rope<CL_F16>(y_dtype, a, grid, s);
  else if (x_dtype == CL_BF16)
    launch_rope<CL_BF16>(y_dtype, a, grid, s);
  else
    launch_rope<CL_F32>(y_dtype, a, grid, s);
  return launched("rope");
}

extern "C" cl_status cl_kv_append(const cl_kv_cache* cache, const void* k, const void* v, int32_t dtype, int32_t tokens,
                                  int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                                  const int32_t* slots, const int32_t* positions, const float* table,
                                  int32_t table_rows, int32_t rot, int32_t layout, void* stream) {
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
  const AppendArgs a = {*cache, {k, v}, {k_token, v_token}, {k_head, v_head}, slots, positions,
                        reinterpret_cast<const float2*>(table), tokens, table ? rot : 0, layout, table_rows};
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
  const unsigned grid = grid_of((int64_t)n * cache->heads * cache->dim);
  if (!grid) return fail(CL_ESIZE, "read: too many slots");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == CL_F16)
    launch_read<CL_F16>(*cache, slots, n, k_out, v_out, grid, s);
  else if (dtype == CL_BF16)
    launch_read<CL_BF16>(*cache, slots, n, k_out, v_out, grid, s);
  else
    launch_read<CL_F32>(*cache, slots, n, k_out, v_out, grid, s);
  return launched("read");
}
