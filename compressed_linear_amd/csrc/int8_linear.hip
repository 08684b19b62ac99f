// int8_linear.hip -- the linear layer in 8-bit integers: rows of values to codes with a scale each, and the product
// of two sets of such rows.
#include <algorithm>

#include "cl_int8.h"
#include "serving.h"

namespace cl {
namespace {

constexpr int kMostK = 131071;  // 128 * 128 * K < 2^31
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
template <int OUT>
__global__ void __launch_bounds__(256) int8_linear_kernel(const int8_t* __restrict__ a, int64_t row, const float* __restrict__ scale, int64_t first,
                                                          int tokens, const int8_t* __restrict__ w, int64_t w_row,
                                                          const float* __restrict__ w_scale, const float* __restrict__ bias, int N, int width,
                                                          typename Elem<OUT>::raw* __restrict__ y, int64_t y_row) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  const int64_t t = first + blockIdx.y;
  if (n >= N) return;
  const int32_t* p = reinterpret_cast<const int32_t*>(a + t * row);
  const int32_t* q = reinterpret_cast<const int32_t*>(w + n * w_row);
  int sum = 0;
  for (int k = 0; k < width / 4; ++k) sum = __builtin_amdgcn_sdot4(p[k], q[k], sum, false);
  float v = (float)sum * scale[t] * w_scale[n];
  if (bias) v += bias[n];
  y[t * y_row + n] = Elem<OUT>::down(v);
}

cl_status check_weights(const int8_t* w, int64_t w_row, const float* w_scale, const float* bias, int N, int K) {
  if (N < 1 || K < 1) return fail(CL_EINVAL, "int8: N >= 1 and K >= 1 are wanted");
  if (K > kMostK) return fail(CL_ESIZE, "int8: K %d above %d", K, kMostK);
  if (!w || !w_scale) return fail(CL_EINVAL, "int8: w or w_scale is NULL");
  if (!aligned_to(w, 16) || !aligned_to(w_scale, 4) || (bias && !aligned_to(bias, 4)))
    return fail(CL_EINVAL, "int8: w must be 16-byte aligned, scales and bias 4-byte");
  if (w_row % 128 || w_row < K) return fail(CL_EINVAL, "int8: rows of %lld bytes for %d codes (a multiple of 128 is wanted)", (long long)w_row, K);
  return CL_OK;
}

cl_status check_codes(const int8_t* codes, int64_t row, const float* scale, int K) {
  if (!codes || !scale) return fail(CL_EINVAL, "int8: codes or scale is NULL");
  if (!aligned_to(codes, 16) || !aligned_to(scale, 4)) return fail(CL_EINVAL, "int8: codes must be 16-byte aligned, scales 4-byte");
  if (row % 128 || row < K) return fail(CL_EINVAL, "int8: rows of %lld bytes for %d codes (a multiple of 128 is wanted)", (long long)row, K);
  return CL_OK;
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

struct Product {
  const int8_t* codes;
  int64_t row;
  const float* scale;
  int tokens;
  const int8_t* w;
  int64_t w_row;
  const float *w_scale, *bias;
  int N, K;
  void* y;
  int64_t y_row;
};

template <int OUT>
void launch_linear(const Product& p, hipStream_t s) {
  for (int64_t first = 0; first < p.tokens; first += 65535)
    hipLaunchKernelGGL((int8_linear_kernel<OUT>), dim3((unsigned)((p.N + 255) / 256), (unsigned)std::min<int64_t>(65535, p.tokens - first)), dim3(256),
                       0, s, p.codes, p.row, p.scale, first, p.tokens, p.w, p.w_row, p.w_scale, p.bias, p.N, (int)padded(p.K),
                       static_cast<typename Elem<OUT>::raw*>(p.y), p.y_row);
}

void launch_linear(const Product& p, int out, hipStream_t s) {
  if (out == CL_F16)
    launch_linear<CL_F16>(p, s);
  else if (out == CL_BF16)
    launch_linear<CL_BF16>(p, s);
  else
    launch_linear<CL_F32>(p, s);
}

}  // namespace
}  // namespace cl

using namespace cl;

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
                                    int32_t y_dtype, int64_t y_row, void* stream) {
  clear_error();
  if (tokens < 0) return fail(CL_EINVAL, "int8: tokens must be >= 0");
  if (tokens == 0) return CL_OK;
  cl_status st = check_weights(w, w_row, w_scale, bias, N, K);
  if (st == CL_OK) st = check_codes(codes, row, scale, K);
  if (st == CL_OK) st = check_output(y, y_dtype);
  if (st != CL_OK) return st;
  launch_linear(Product{codes, row, scale, tokens, w, w_row, w_scale, bias, N, K, y, y_row}, y_dtype, static_cast<hipStream_t>(stream));
  return launched("int8 linear");
}

extern "C" size_t cl_int8_work_bytes(int32_t tokens, int32_t K) {
  if (tokens < 1 || K < 1 || K > kMostK) return 0;
  return (size_t)tokens * (padded(K) + 4);
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
  const size_t need = cl_int8_work_bytes(tokens, K);
  if (work_bytes < need) return fail(CL_ENOMEM, "int8: the workspace has %zu bytes, %zu are wanted", work_bytes, need);
  if (need && (!work || !aligned_to(work, 16))) return fail(CL_EINVAL, "int8: work is NULL or misaligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  int8_t* codes = static_cast<int8_t*>(work);
  float* scale = reinterpret_cast<float*>(codes + (size_t)tokens * padded(K));
  launch_quant(x, dtype, x_row, tokens, K, clamp, codes, padded(K), scale, s);
  launch_linear(Product{codes, padded(K), scale, tokens, w, w_row, w_scale, bias, N, K, y, y_row}, y_dtype, s);
  return launched("int8 forward");
}
