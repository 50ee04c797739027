// Operands of the 8-bit floating-point product: matrices rounded to e4m3 with a scale per block of 128
// columns, and packed GPTQ codes turned into e4m3 integers with the grids' own scales.
//
// Rounding.  The scale of a block is the smallest power of two s with max|x| <= 448 s, read off the
// exponent and the mantissa of the maximum (448 = 1.75 * 2^8), so x / s is exact and the conversion to
// e4m3 is the only rounding.  Both kernels here move bytes and do little else: the bound is HBM.
#include <algorithm>

#include "kernels.h"
#include "common.cuh"

namespace gptq {
namespace {

constexpr int kBlockCols = 128;  // columns per scale
constexpr int kThreads = 256;

// e4m3 codes of (lo, hi): rounded to nearest even, saturated at 448, NaN kept
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ bool is_finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// exponent e of the scale 2^e for a block maximum (see the header comment), >= -126
__device__ __forceinline__ int scale_exponent(float amax) {
  if (amax == 0.0f) return 0;
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, -126);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// eight consecutive values as fp32 (16-byte aligned)
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its fp32
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ float finite_amax8(const float (&v)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, is_finite(v[i]) ? fabsf(v[i]) : 0.0f);
  return a;
}

// eight codes of v * inv; NaN and infinities become NaN
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = is_finite(v[i]) ? v[i] * inv : __uint_as_float(0x7FC00000u);
  return make_uint2(cvt_e4m3x2(s[0], s[1]) | (cvt_e4m3x2(s[2], s[3]) << 16),
                    cvt_e4m3x2(s[4], s[5]) | (cvt_e4m3x2(s[6], s[7]) << 16));
}

// One scale per row and 128 columns: 16 lanes hold a block, eight values each.  A CTA takes `rows_per`
// rows at a time with kThreads / rows_per threads on each (a power of two >= 16).
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_rows_kernel(const T* __restrict__ X, int64_t m, int k, int kb,
                                                                     int rows_per, uint8_t* __restrict__ Q,
                                                                     float* __restrict__ scales) {
  const int per_row = kThreads / rows_per;
  const int sub = threadIdx.x / per_row, t = threadIdx.x % per_row;
  const int granules = kb * 16;  // 8-column granules of a row, the last block filled up
  for (int64_t r = (int64_t)blockIdx.x * rows_per + sub; r - sub < m; r += (int64_t)gridDim.x * rows_per) {
    const bool row_ok = r < m;
    const T* src = X + r * k;
    for (int c0 = 0; c0 < granules; c0 += per_row) {  // the same trips for every lane: the shuffles need all of them
      const int c = c0 + t;
      const bool ok = row_ok && c * 8 < k;
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (ok) load8<T>(src + c * 8, v);
      float a = finite_amax8(v);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      const int e = scale_exponent(a);
      if (ok) *reinterpret_cast<uint2*>(Q + r * k + c * 8) = codes8(v, pow2f(-e));
      if (row_ok && (c & 15) == 0 && c < granules) scales[r * kb + (c >> 4)] = pow2f(e);
    }
  }
}

// One scale per 128 x 128 block: one CTA per block, 16 threads across the columns, 16 rows per pass.
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_blocks_kernel(const T* __restrict__ X, int64_t m, int k,
                                                                       int kb, uint8_t* __restrict__ Q,
                                                                       float* __restrict__ scales) {
  __shared__ float warp_max_of[kThreads / 32];
  const int64_t rb = blockIdx.x / kb;
  const int cb = blockIdx.x % kb;
  const int col = cb * kBlockCols + (threadIdx.x & 15) * 8;
  const int64_t r0 = rb * 128 + (threadIdx.x >> 4);
  float v[8][8];
  float a = 0.0f;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
    if (r0 + 16 * p < m && col < k) load8<T>(X + (r0 + 16 * p) * k + col, v[p]);
  }
#pragma unroll
  for (int p = 0; p < 8; ++p) a = fmaxf(a, finite_amax8(v[p]));
  a = warp_max(a);
  if ((threadIdx.x & 31) == 0) warp_max_of[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) a = fmaxf(a, warp_max_of[w]);
  const int e = scale_exponent(a);
  const float inv = pow2f(-e);
#pragma unroll
  for (int p = 0; p < 8; ++p)
    if (r0 + 16 * p < m && col < k) *reinterpret_cast<uint2*>(Q + (r0 + 16 * p) * k + col) = codes8(v[p], inv);
  if (threadIdx.x == 0) scales[rb * kb + cb] = pow2f(e);
}

// A thread turns one unit of 32 codes (BITS words) into 32 e4m3 integers q - zero.  1 + q 2^-b is formed
// by masking the code into a mantissa; one FMA then gives q - zero exactly.
template <int BITS>
__global__ void __launch_bounds__(kThreads) fp8_from_packed_kernel(const uint32_t* __restrict__ packed,
                                                                   const float* __restrict__ scales,
                                                                   const int32_t* __restrict__ zeros, int64_t m,
                                                                   int units, int group_units, int ng,
                                                                   uint8_t* __restrict__ Q,
                                                                   float* __restrict__ scales_out) {
  constexpr int P = 23 - BITS;
  const int kb = (units + 3) >> 2;
  for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < m * units;
       e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = e / units;
    const int u = (int)(e - r * units);
    uint32_t w[BITS];
#pragma unroll
    for (int i = 0; i < BITS; ++i) w[i] = __ldg(packed + e * BITS + i);
    const int64_t grid = r * ng + u / group_units;
    const float offset = -(float)(1 << BITS) - (float)__ldg(zeros + grid);
    uint32_t out[8];
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int bit = BITS * (j + h), word = bit >> 5, s = bit & 31;
        uint32_t v;
        if (s >= P)
          v = __funnelshift_r(w[word], word + 1 < BITS ? w[word + 1] : 0u, s - P);
        else
          v = w[word] << (P - s);  // s + BITS < 23: the code ends inside its word
        f[h] = fmaf(__uint_as_float((v & (((1u << BITS) - 1u) << P)) | 0x3F800000u), (float)(1 << BITS), offset);
      }
      const uint32_t c = cvt_e4m3x2(f[0], f[1]);
      if (j % 4 == 0) out[j / 4] = c; else out[j / 4] |= c << 16;
    }
    uint4* dst = reinterpret_cast<uint4*>(Q + e * 32);
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    if ((u & 3) == 0) scales_out[r * kb + (u >> 2)] = __ldg(scales + grid);
  }
}

template <typename T>
gptq_status quantize_typed(const T* X, int64_t m, int k, int block_rows, uint8_t* Q, float* scales, cudaStream_t s) {
  const int kb = (k + kBlockCols - 1) / kBlockCols;
  if (block_rows == 1) {
    int per_row = 16;
    while (per_row < kThreads && per_row < kb * 16) per_row *= 2;
    const int rows_per = kThreads / per_row;
    const int64_t blocks = std::min<int64_t>((m + rows_per - 1) / rows_per, 148 * 16);
    fp8_quantize_rows_kernel<T><<<(unsigned)blocks, kThreads, 0, s>>>(X, m, k, kb, rows_per, Q, scales);
  } else {
    const int64_t blocks = (m + 127) / 128 * kb;
    if (blocks > 0x7fffffff) return GPTQ_ERR_ARG;
    fp8_quantize_blocks_kernel<T><<<(unsigned)blocks, kThreads, 0, s>>>(X, m, k, kb, Q, scales);
  }
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace

gptq_status fp8_quantize_launch(const void* X, int32_t x_dtype, int64_t m, int64_t k, int32_t block_rows, void* Q,
                                float* scales, cudaStream_t stream) {
  uint8_t* q = static_cast<uint8_t*>(Q);
  switch (x_dtype) {
    case GPTQ_BF16: return quantize_typed(static_cast<const __nv_bfloat16*>(X), m, (int)k, block_rows, q, scales, stream);
    case GPTQ_FP16: return quantize_typed(static_cast<const __half*>(X), m, (int)k, block_rows, q, scales, stream);
    default: return quantize_typed(static_cast<const float*>(X), m, (int)k, block_rows, q, scales, stream);
  }
}

gptq_status fp8_from_packed_launch(const int32_t* packed, const float* scales, const int32_t* zeros, int64_t m,
                                   int64_t k, int32_t bits, int32_t group_size, void* Q, float* scales_out,
                                   cudaStream_t stream) {
  const uint32_t* pw = reinterpret_cast<const uint32_t*>(packed);
  uint8_t* q = static_cast<uint8_t*>(Q);
  const int units = (int)(k / 32), gu = group_size ? group_size / 32 : units, ng = group_size ? (int)(k / group_size) : 1;
  const unsigned blocks = (unsigned)std::min<int64_t>((m * units + kThreads - 1) / kThreads, 148 * 16);
  switch (bits) {
    case 2: fp8_from_packed_kernel<2><<<blocks, kThreads, 0, stream>>>(pw, scales, zeros, m, units, gu, ng, q, scales_out); break;
    case 3: fp8_from_packed_kernel<3><<<blocks, kThreads, 0, stream>>>(pw, scales, zeros, m, units, gu, ng, q, scales_out); break;
    default: fp8_from_packed_kernel<4><<<blocks, kThreads, 0, stream>>>(pw, scales, zeros, m, units, gu, ng, q, scales_out); break;
  }
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
