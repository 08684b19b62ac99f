// serving.h -- helpers shared by the operators of include/cl_serving.h:
// 16- and 32-bit element types and host checks.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cl_serving.h"
#include "internal.h"

namespace cl {

// Element types by cl_dtype.  Conversions to 16 bits round to nearest-even once.
template <int DT>
struct Elem;
template <>
struct Elem<CL_F16> {
  typedef uint16_t raw;
  static __device__ __forceinline__ float up(raw b) { return (float)__builtin_bit_cast(_Float16, b); }
  static __device__ __forceinline__ raw down(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
};
template <>
struct Elem<CL_BF16> {
  typedef uint16_t raw;
  static __device__ __forceinline__ float up(raw b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
  static __device__ __forceinline__ raw down(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};
template <>
struct Elem<CL_F32> {
  typedef float raw;
  static __device__ __forceinline__ float up(raw b) { return b; }
  static __device__ __forceinline__ raw down(float f) { return f; }
};

typedef float v4 __attribute__((ext_vector_type(4)));
typedef uint32_t w4 __attribute__((ext_vector_type(4)));
typedef uint32_t w2 __attribute__((ext_vector_type(2)));
typedef _Float16 half_pair __attribute__((ext_vector_type(2)));
typedef __bf16 bf16_pair __attribute__((ext_vector_type(2)));

// Two values rounded to 16 bits, in one word.
template <int DT>
__device__ __forceinline__ uint32_t down2(float x, float y) {
  if constexpr (DT == CL_F16)
    return __builtin_bit_cast(uint32_t, half_pair{(_Float16)x, (_Float16)y});
  else
    return __builtin_bit_cast(uint32_t, bf16_pair{(__bf16)x, (__bf16)y});
}

// Eight contiguous elements, 16-byte aligned.
template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::raw* p, float (&v)[8]) {
  if constexpr (DT == CL_F32) {
    const v4* q = reinterpret_cast<const v4*>(p);
    const v4 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const w4 a = *reinterpret_cast<const w4*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<DT>::up((uint16_t)(a[i / 2] >> (16 * (i % 2))));
  }
}
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::raw* p, const float (&v)[8]) {
  if constexpr (DT == CL_F32) {
    v4* q = reinterpret_cast<v4*>(p);
    q[0] = v4{v[0], v[1], v[2], v[3]};
    q[1] = v4{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<w4*>(p) = w4{down2<DT>(v[0], v[1]), down2<DT>(v[2], v[3]), down2<DT>(v[4], v[5]), down2<DT>(v[6], v[7])};
  }
}

inline size_t elem_size(int dtype) { return dtype == CL_F32 ? 4 : 2; }
inline bool elem_ok(int dtype) { return dtype == CL_F16 || dtype == CL_BF16 || dtype == CL_F32; }
inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A cache description that the kernels may trust; `dim_of_attention`: dim has to be 64 or 128.
inline cl_status check_cache(const cl_kv_cache* c) {
  if (!c) return fail(CL_EINVAL, "cache is NULL");
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(CL_EINVAL, "cache: a pointer is NULL");
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(c->k_scale, 8) || !aligned_to(c->v_scale, 8))
    return fail(CL_EINVAL, "cache: k and v must be 16-byte aligned, scales 8-byte aligned");
  if (c->kind != CL_KV_INT8 && c->kind != CL_KV_INT4) return fail(CL_EINVAL, "cache: unknown kind %d", c->kind);
  if (c->pages < 1 || c->heads < 1 || c->page_size < 1) return fail(CL_EINVAL, "cache: sizes must be >= 1");
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return fail(CL_EINVAL, "cache: page_size %d is no power of two in [16, 1024]", c->page_size);
  if (c->dim != 64 && c->dim != 128) return fail(CL_EUNSUPPORTED, "cache: dim %d (64 and 128 are built)", c->dim);
  if (c->heads > 65535) return fail(CL_ESIZE, "cache: more than 65535 heads");
  if ((int64_t)c->pages * c->page_size >= ((int64_t)1 << 31)) return fail(CL_ESIZE, "cache: 2^31 slots or more");
  return CL_OK;
}

// Rotation arguments, where there is a table.
inline cl_status check_rope(const int32_t* positions, const float* table, int table_rows, int rot, int layout, int dim) {
  if (!positions || !table) return fail(CL_EINVAL, "rope: positions or table is NULL");
  if (!aligned_to(positions, 4) || !aligned_to(table, 8)) return fail(CL_EINVAL, "rope: positions or table is misaligned");
  if (table_rows < 1) return fail(CL_EINVAL, "rope: the table has no rows");
  if (rot < 2 || rot % 2 || rot > dim) return fail(CL_EINVAL, "rope: rot %d is odd or not in [2, %d]", rot, dim);
  if (layout != CL_ROPE_HALF && layout != CL_ROPE_INTERLEAVED) return fail(CL_EINVAL, "rope: unknown layout %d", layout);
  return CL_OK;
}

// Whether every head of a tensor starts on a 16-byte boundary.
inline bool heads_aligned(const void* p, int dtype, int64_t token, int64_t head) {
  const int64_t e = (int64_t)elem_size(dtype);
  return aligned_to(p, 16) && token * e % 16 == 0 && head * e % 16 == 0;
}

// A launch holds fewer than 2^32 threads along a dimension (the runtime drops the rest without an error), so longer work goes
// in pieces: f(first, count) over n tokens (rows) of `each` threads in workgroups of at most 1024, where one token fits.
constexpr int64_t kLaunch = ((int64_t)1 << 32) - 1024;
template <typename F>
void in_pieces(int64_t n, int64_t each, F f) {
  const int64_t most = kLaunch / each;
  for (int64_t at = 0; at < n; at += most) f(at, n - at < most ? n - at : most);
}

// An address `n` elements on.
inline const void* beyond(const void* p, int dtype, int64_t n) { return static_cast<const uint8_t*>(p) + n * (int64_t)elem_size(dtype); }
inline void* beyond(void* p, int dtype, int64_t n) { return static_cast<uint8_t*>(p) + n * (int64_t)elem_size(dtype); }

inline cl_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? CL_OK : fail(CL_EHIP, "%s: launch failed: %s", what, hipGetErrorString(e));
}

// (y1, y2) of a pair, each product and sum rounded to fp32 (no fused multiply-add), so that a plain
// fp32 evaluation of the formula gives the same bits.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
#pragma clang fp contract(off)
  const float y1 = a * c - b * s;
  const float y2 = b * c + a * s;
  a = y1;
  b = y2;
}

}  // namespace cl
