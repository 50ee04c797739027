// Operands of the 8-bit floating-point product: matrices rounded to e4m3 with a scale per block of 128
// columns, and packed GPTQ codes turned into e4m3 integers with the grids' own scales.
//
// Rounding.  The scale of a block is the smallest power of two s with max|x| <= 448 s, read off the
// exponent and the mantissa of the maximum (448 = 1.75 * 2^8), so x / s is exact and the conversion to
// e4m3 is the only rounding.  Both kernels here move bytes and do little else: the bound is HBM.
#include <algorithm>
#include <type_traits>

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

// Eight consecutive values as they lie in memory (16-byte aligned), their largest magnitude as an ordered
// integer (an fp32's bits: magnitudes compare like their bits, infinities and NaN above all), their codes.
template <typename T>
struct Granule {
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
      return i & 1 ? f.y : f.x;
    } else {  // a bf16 is the upper half of its fp32
      return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    const uint32_t h = max(m & 0xFFFFu, m >> 16);
    if constexpr (std::is_same<T, __half>::value)
      return h >= 0x7C00u ? 0x7F800000u : __float_as_uint(__half2float(__ushort_as_half((uint16_t)h)));
    else
      return h << 16;
  }
};
template <>
struct Granule<float> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* p) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0;
  }
  __device__ __forceinline__ float value(int i) const { return __uint_as_float(w[i]); }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    return m;
  }
};

constexpr uint32_t kInfBits = 0x7F800000u;

template <typename T>
__device__ __forceinline__ uint2 codes8(const Granule<T>& v, float inv) {
  return make_uint2(cvt_e4m3x2(v.value(0) * inv, v.value(1) * inv) | (cvt_e4m3x2(v.value(2) * inv, v.value(3) * inv) << 16),
                    cvt_e4m3x2(v.value(4) * inv, v.value(5) * inv) | (cvt_e4m3x2(v.value(6) * inv, v.value(7) * inv) << 16));
}

// the same for a block with infinities or NaN in it: the largest finite magnitude, and codes with NaN for both
template <typename T>
__device__ __noinline__ uint32_t finite_top(const Granule<T>& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v.value(i)) & 0x7FFFFFFFu;
    m = max(m, b < kInfBits ? b : 0u);
  }
  return m;
}
template <typename T>
__device__ __noinline__ uint2 finite_codes8(const Granule<T>& v, float inv) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = is_finite(v.value(i)) ? v.value(i) * inv : __uint_as_float(0x7FC00000u);
  return make_uint2(cvt_e4m3x2(s[0], s[1]) | (cvt_e4m3x2(s[2], s[3]) << 16),
                    cvt_e4m3x2(s[4], s[5]) | (cvt_e4m3x2(s[6], s[7]) << 16));
}

__device__ __forceinline__ uint32_t max16(uint32_t v) {  // over the 16 lanes of a block
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// One scale per row and 128 columns: 16 lanes hold a block, eight values each (all lanes call it).
template <typename T>
__device__ __forceinline__ void quantize_granule(const Granule<T>& v, bool ok, uint8_t* q, float* scale, bool first) {
  uint32_t top = max16(v.top());
  const bool odd = top >= kInfBits;
  if (__any_sync(0xffffffffu, odd)) {
    const uint32_t f = max16(finite_top(v));
    if (odd) top = f;
  }
  const int e = scale_exponent(__uint_as_float(top));
  if (ok) *reinterpret_cast<uint2*>(q) = odd ? finite_codes8(v, pow2f(-e)) : codes8(v, pow2f(-e));
  if (first) *scale = pow2f(e);
}

// Rows of whole blocks (k % 128 == 0): blocks lie one behind the other, whatever the row.  Every thread has four
// independent granules in flight: 16384 x 11008 bf16 in rows of their own took 146 us with one, 101 with four (5.4
// TB/s; bound by HBM).
constexpr int kInFlight = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_linear_kernel(const T* __restrict__ X, int64_t granules,
                                                                       uint8_t* __restrict__ Q,
                                                                       float* __restrict__ scales) {
  const int64_t g0 = (int64_t)blockIdx.x * (kThreads * kInFlight) + threadIdx.x;
  Granule<T> v[kInFlight];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) {
    v[i].clear();
    if (g0 + i * kThreads < granules) v[i].load(X + (g0 + i * kThreads) * 8);
  }
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) {
    const int64_t g = g0 + i * kThreads;
    const bool ok = g < granules;
    quantize_granule<T>(v[i], ok, Q + g * 8, scales + (g >> 4), ok && (g & 15) == 0);
  }
}

// Other rows: a CTA takes `rows_per` rows at a time with kThreads / rows_per threads on each (a power of two >= 16).
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_rows_kernel(const T* __restrict__ X, int64_t m, int k, int kb,
                                                                     int rows_per, uint8_t* __restrict__ Q,
                                                                     float* __restrict__ scales) {
  const int per_row = kThreads / rows_per;
  const int sub = threadIdx.x / per_row, t = threadIdx.x % per_row;
  const int granules = kb * 16;  // 8-column granules of a row, the last block filled up
  for (int64_t r = (int64_t)blockIdx.x * rows_per + sub; r - sub < m; r += (int64_t)gridDim.x * rows_per) {
    const bool row_ok = r < m;
    for (int c0 = 0; c0 < granules; c0 += per_row) {  // the same trips for every lane: the shuffles need all of them
      const int c = c0 + t;
      const bool ok = row_ok && c * 8 < k;
      Granule<T> v;
      v.clear();
      if (ok) v.load(X + r * k + c * 8);
      quantize_granule<T>(v, ok, Q + r * k + c * 8, scales + r * kb + (c >> 4), row_ok && (c & 15) == 0 && c < granules);
    }
  }
}

// One scale per 128 x 128 block: one CTA per block, 16 threads across the columns, 16 rows per pass.
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_blocks_kernel(const T* __restrict__ X, int64_t m, int k,
                                                                       int kb, uint8_t* __restrict__ Q,
                                                                       float* __restrict__ scales) {
  __shared__ uint32_t tops[2][kThreads / 32];
  const int64_t rb = blockIdx.x / kb;
  const int cb = blockIdx.x % kb;
  const int col = cb * kBlockCols + (threadIdx.x & 15) * 8;
  const int64_t r0 = rb * 128 + (threadIdx.x >> 4);
  Granule<T> v[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    v[p].clear();
    if (r0 + 16 * p < m && col < k) v[p].load(X + (r0 + 16 * p) * k + col);
  }
  auto block_max = [&](uint32_t a, uint32_t* of) {
    a = __reduce_max_sync(0xffffffffu, a);
    if ((threadIdx.x & 31) == 0) of[threadIdx.x >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) a = max(a, of[w]);
    return a;
  };
  uint32_t a = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p) a = max(a, v[p].top());
  uint32_t top = block_max(a, tops[0]);
  const bool odd = top >= kInfBits;  // the same for the whole CTA
  if (odd) {
    a = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) a = max(a, finite_top(v[p]));
    top = block_max(a, tops[1]);
  }
  const int e = scale_exponent(__uint_as_float(top));
  const float inv = pow2f(-e);
#pragma unroll
  for (int p = 0; p < 8; ++p)
    if (r0 + 16 * p < m && col < k)
      *reinterpret_cast<uint2*>(Q + (r0 + 16 * p) * k + col) = odd ? finite_codes8(v[p], inv) : codes8(v[p], inv);
  if (threadIdx.x == 0) scales[rb * kb + cb] = pow2f(e);
}

// Eight codes of a unit (codes 8 k .. 8 k + 7) as nibbles of a word, code 8 k in the lowest.  Narrower codes are spread
// in three steps that each move the upper half of a field up.
template <int BITS>
__device__ __forceinline__ uint32_t nibbles(const uint32_t (&w)[BITS], int k) {
  if constexpr (BITS == 4) {
    return w[k];
  } else if constexpr (BITS == 3) {  // bits 24 k .. 24 k + 23 of the unit
    uint32_t x = k == 0 ? w[0] : (k == 3 ? w[2] >> 8 : __funnelshift_r(w[k - 1], w[k], k == 1 ? 24 : 16));
    x = (x & 0x00000FFFu) | ((x << 4) & 0x0FFF0000u);
    x = (x & 0x003F003Fu) | ((x << 2) & 0x3F003F00u);
    return (x & 0x07070707u) | ((x << 1) & 0x70707070u);
  } else {
    uint32_t x = k & 1 ? w[k >> 1] >> 16 : w[k >> 1];
    x = (x & 0x000000FFu) | ((x << 8) & 0x00FF0000u);
    x = (x & 0x000F000Fu) | ((x << 4) & 0x0F000F00u);
    return (x & 0x03030303u) | ((x << 2) & 0x30303030u);
  }
}

// A thread turns one unit of 32 codes (BITS words) into 32 e4m3 integers q - zero: the bytes for q = 0 .. 2^b - 1 come
// from a table by zero point, and a byte permutation with the codes as selectors picks four at a time (two
// and a blend at 4 bits, where the top bit chooses the half of the table).  One instruction or two a code; masking,
// one FMA and a conversion per code took 17.5 us for 11008 x 4096 codes of 4 bits, this 14.9 (4.6 TB/s).  Zero
// points outside the grid take that way.
template <int BITS>
__global__ void __launch_bounds__(kThreads) fp8_from_packed_kernel(const uint32_t* __restrict__ packed,
                                                                   const float* __restrict__ scales,
                                                                   const int32_t* __restrict__ zeros, int64_t n,
                                                                   int units, int group_units, int ng,
                                                                   uint8_t* __restrict__ Q,
                                                                   float* __restrict__ scales_out) {
  constexpr int P = 23 - BITS;
  __shared__ __align__(16) uint8_t table[16][16];  // [zero][code]
  static_assert(kThreads == 256, "an entry per thread");
  table[threadIdx.x >> 4][threadIdx.x & 15] = (uint8_t)cvt_e4m3x2((float)((int)(threadIdx.x & 15) - (int)(threadIdx.x >> 4)), 0.0f);
  __syncthreads();
  const int kb = (units + 3) >> 2;
  for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = n <= 0x7fffffff ? (int64_t)((uint32_t)e / (uint32_t)units) : e / units;
    const int u = (int)(e - r * units);
    uint32_t w[BITS];
    if (BITS == 4 && (reinterpret_cast<uintptr_t>(packed) & 15) == 0) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(packed) + e);
      w[0] = v.x, w[1] = v.y, w[2 % BITS] = v.z, w[3 % BITS] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < BITS; ++i) w[i] = __ldg(packed + e * BITS + i);
    }
    const int64_t grid = r * ng + (ng == 1 ? 0 : u / group_units);
    const int32_t z = __ldg(zeros + grid);
    uint32_t out[8];
    if ((uint32_t)z < 16u) {
      const uint4 t = *reinterpret_cast<const uint4*>(table[z]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t c = nibbles<BITS>(w, k);
        if constexpr (BITS == 4) {
          const uint32_t low = c & 0x77777777u, top = (c >> 3) & 0x11111111u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t s = h ? low >> 16 : low, f = __byte_perm(0x0000FF00u, 0u, h ? top >> 16 : top);
            out[2 * k + h] = (__byte_perm(t.x, t.y, s) & ~f) | (__byte_perm(t.z, t.w, s) & f);
          }
        } else {
          out[2 * k] = __byte_perm(t.x, t.y, c), out[2 * k + 1] = __byte_perm(t.x, t.y, c >> 16);
        }
      }
    } else {
      const float offset = -(float)(1 << BITS) - (float)z;
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
  const int64_t granules = m * (k / 8), linear_blocks = (granules + kThreads * kInFlight - 1) / (kThreads * kInFlight);
  if (block_rows == 1 && k % kBlockCols == 0 && linear_blocks <= 0x7fffffff) {
    fp8_quantize_linear_kernel<T><<<(unsigned)linear_blocks, kThreads, 0, s>>>(X, granules, Q, scales);
  } else if (block_rows == 1) {
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
    case 2: fp8_from_packed_kernel<2><<<blocks, kThreads, 0, stream>>>(pw, scales, zeros, m * units, units, gu, ng, q, scales_out); break;
    case 3: fp8_from_packed_kernel<3><<<blocks, kThreads, 0, stream>>>(pw, scales, zeros, m * units, units, gu, ng, q, scales_out); break;
    default: fp8_from_packed_kernel<4><<<blocks, kThreads, 0, stream>>>(pw, scales, zeros, m * units, units, gu, ng, q, scales_out); break;
  }
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
