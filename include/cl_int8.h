/*
 * cl_int8.h -- C ABI of the linear layer in 8-bit integers on MI355X (gfx950): weights with a scale to each output
 * channel, activations quantised on the way in with a scale to each token, products summed exactly in
 * 32-bit integers.
 *
 *     y[t, n] = (sum_k a[t, k] w[n, k]) * s[t] * w_scale[n] + bias[n]
 *
 * Conventions are those of cl_serving.h: status codes, caller-owned device pointers, streams as void*, work asynchronous
 * on the stream, nothing allocated, every entry recordable into a HIP graph, cl_dtype for element types, strides in
 * elements.  A call with no rows returns CL_OK and launches nothing.
 *
 * Codes lie in rows of `row` bytes, a multiple of 128, at least K and at most 2^23; a row's bytes from K to the next
 * multiple of 128 are readable, and zeros in weights.  Codes are 16-byte aligned.
 */
#ifndef CL_INT8_H
#define CL_INT8_H

#include "cl_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * cl_int8_quant -- rows of values to codes and a scale: activations by token, or weights by output channel.  With
 * v = x, or x clamped to [-clamp, clamp] where clamp > 0, and a = max_k |v[k]| of a row
 *     scale = a * (1 / 127)        code = rint(v * (1 / scale))
 * every constant, product and quotient an fp32 value, rounded to nearest-even.  A row with a < 2^-100 has scale 0
 * and codes 0; one with a NaN or an infinity (after the clamp) has scale NaN and codes 0, so that its outputs are NaN.
 *   x, dtype         device, [rows, K], row stride x_row
 *   codes, row       device, [rows, row] int8: K codes, then zeros up to the next multiple of 128
 *   scale            device, [rows] fp32
 * Errors: CL_EINVAL (sizes, unknown type, NULL or misaligned pointers, clamp negative or not finite), CL_ESIZE (K > 131071), CL_EHIP.
 */
cl_status cl_int8_quant(const void* x, int32_t dtype, int64_t x_row, int32_t rows, int32_t K, float clamp, int8_t* codes,
                        int64_t row, float* scale, void* stream);

/*
 * cl_int8_linear -- the product with activations that are codes already.
 *   codes, row, scale    device, [tokens, row] int8 and [tokens] fp32, as cl_int8_quant leaves them (any int8 will do)
 *   w, w_row, w_scale    device, [N, w_row] int8 and [N] fp32
 *   bias                 device, [N] fp32, or NULL
 *   y, y_dtype, y_row    device, [tokens, N], row stride y_row; the sum of products is rounded to fp32, then each product
 *                        with a scale and the sum with the bias, then the result to y's type
 *   work                 device, cl_int8_work_bytes(tokens, N, K, 1) bytes, 16-byte aligned (may be NULL where that is 0);
 *                        it is this call's alone until the call has run
 * K <= 131071, so that no sum of products of two int8 passes 32 bits; N <= 2^25.  A row's outputs do not depend on the other rows, nor
 * on how many there are.
 * Errors: CL_EINVAL, CL_ESIZE, CL_ENOMEM (work_bytes too small), CL_EHIP.
 */
size_t cl_int8_work_bytes(int32_t tokens, int32_t N, int32_t K, int32_t quantised);
cl_status cl_int8_linear(const int8_t* codes, int64_t row, const float* scale, int32_t tokens, const int8_t* w,
                         int64_t w_row, const float* w_scale, const float* bias, int32_t N, int32_t K, void* y,
                         int32_t y_dtype, int64_t y_row, void* work, size_t work_bytes, void* stream);

/*
 * cl_int8_forward -- cl_int8_quant and cl_int8_linear in one call.
 *   work             device, cl_int8_work_bytes(tokens, N, K, 0) bytes, as for cl_int8_linear
 * Errors: as both.
 */
cl_status cl_int8_forward(const void* x, int32_t dtype, int64_t x_row, int32_t tokens, float clamp, const int8_t* w,
                          int64_t w_row, const float* w_scale, const float* bias, int32_t N, int32_t K, void* y,
                          int32_t y_dtype, int64_t y_row, void* work, size_t work_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif
