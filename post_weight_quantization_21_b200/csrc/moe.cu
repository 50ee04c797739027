// A mixture-of-experts layer for a few tokens over packed weights: router, the chosen experts' gate / up
// products, the activation, the down product and the weighted sum.
//   l = x R^T,  p = softmax(l),  e_1 .. e_K = the K largest p,  w_i = p[e_i] (over their sum when renormalised)
//   y = sum_i w_i D_{e_i} a_i,   a_i = silu(G_{e_i} x) * (U_{e_i} x)  or  relu(U_{e_i} x)
// with every matrix What[r, j] = scale[r, g] (q[r, j] - zero[r, g]) read as packed codes.
//
// The bytes of the chosen experts' codes are the floor, so the work to keep below HBM's time is taking the
// codes apart.  A code masked in place into the low bits of an fp16 is a subnormal, q 2^(p - 24) exactly:
// one AND for two codes, nothing to subtract, and the pair is a ready fragment of mma.m16n8k16 (weights on
// the M side, up to 8 tokens on the N side: a product with so few columns is no tcgen05 shape, and the tensor
// pipe has time to spare here).  The order of the columns in a sum is free, so a pair is two codes that lie
// 16 bits apart (see Pairs) and the tokens' values are laid out to match, multiplied by 2^-p.  The
// zero point leaves the sum as zero * sum_j x_j, which starts the accumulator: sum_j (q_j - zero) x_j = sum q x -
// zero sum x.  Products are aligned by their operands' exponents before they are added, and a subnormal's
// exponent says 2^-14 whatever its size, so sums over subnormals keep some seven bits less than they could:
// results off by 1e-5 to 4e-5, a tenth of fp16's own rounding and less.  For an fp32 Y the codes are therefore
// joined with the exponent of 1024 and 1024 + zero 2^p is taken off, which leaves (q - zero) 2^p as a normal
// fp16, exactly: one subtraction more per pair.
//
// Tokens become fp16 terms of x 2^-e, e per token and 128 columns so that the largest value lies below 2^15: one
// term holds a bf16 or fp16 value exactly as long as it is not below 2^-21 of the block's largest (then it is off
// by less than 2^-32 of that), two terms hold an fp32 value to 2^-24 of itself.  The intermediate a_i, kept in fp32,
// takes two terms, or one where Y is bf16 (2^-12 beside the result's own 2^-9).  Products are then exact in
// the tensor core, sums run there over 128 columns and in fp32 beyond.
//
// Launches: router logits and the tokens' layout; top-K and the lists of tokens per expert (one launch with the
// router where there are few logits); the up product
// with the activation; the activations' layout; the down product; the weighted sum in the order of the choice.
// No atomics: results are deterministic.
#include <algorithm>

#include "kernels.h"
#include "common.cuh"

namespace gptq {
namespace {

constexpr int kMaxExperts = 256;
constexpr int kMaxTopK = 16;
constexpr int kMaxTokens = 64;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;

// ------------------------------------------------------------------ columns of a unit of 32 codes
// Register i of a unit holds columns lo(i) and hi(i) in its halves, both at bit p(i).
template <int BITS>
struct Pairs;
template <>
struct Pairs<4> {  // register 4 w + 2 h + s: word w shifted by 8 h, masked at bit 4 s
  __host__ __device__ static constexpr int lo(int i) { return 8 * (i / 4) + i % 4; }
  __host__ __device__ static constexpr int hi(int i) { return lo(i) + 4; }
  __host__ __device__ static constexpr int p(int i) { return 4 * (i & 1); }
};
template <>
struct Pairs<2> {  // register 8 w + s: word w, shifted by 10 from s = 5 on
  __host__ __device__ static constexpr int lo(int i) { return 16 * (i / 8) + i % 8; }
  __host__ __device__ static constexpr int hi(int i) { return lo(i) + 8; }
  __host__ __device__ static constexpr int p(int i) { return 2 * (i % 8 % 5); }
};
template <>
struct Pairs<3> {  // registers 5 b + s: two runs of five codes side by side; register 15: the codes across words
  __host__ __device__ static constexpr int lo(int i) { return i == 15 ? 10 : (i < 10 ? i : i + 12); }
  __host__ __device__ static constexpr int hi(int i) { return i == 15 ? 21 : (i < 10 ? i + 11 : i + 17); }
  __host__ __device__ static constexpr int p(int i) { return i == 15 ? 0 : 3 * (i % 5 % 3); }
};
template <int BITS>
__host__ __device__ constexpr bool pairs_ok() {
  uint32_t seen = 0;
  for (int i = 0; i < 16; ++i) {
    seen |= 1u << Pairs<BITS>::lo(i) | 1u << Pairs<BITS>::hi(i);
    if (Pairs<BITS>::p(i) + BITS > 10) return false;  // a subnormal's mantissa
  }
  return seen == 0xffffffffu;  // every column once
}
static_assert(pairs_ok<2>() && pairs_ok<3>() && pairs_ok<4>(), "column order");

template <int BITS, int P>
__device__ __forceinline__ uint32_t mask_pair(uint32_t v) {
  constexpr uint32_t m = ((1u << BITS) - 1u) << P;
  return v & (m | (m << 16));
}

// registers 4 q .. 4 q + 3 of a unit: codes q 2^(p - 24) in both halves (q a constant once unrolled)
template <int BITS>
__device__ __forceinline__ void unit_quad(const uint32_t (&w)[BITS], int q, uint32_t (&v)[4]);
template <>
__device__ __forceinline__ void unit_quad<4>(const uint32_t (&w)[4], int q, uint32_t (&v)[4]) {
  const uint32_t b = w[q] >> 8;
  v[0] = mask_pair<4, 0>(w[q]), v[1] = mask_pair<4, 4>(w[q]), v[2] = mask_pair<4, 0>(b), v[3] = mask_pair<4, 4>(b);
}
template <>
__device__ __forceinline__ void unit_quad<2>(const uint32_t (&w)[2], int q, uint32_t (&v)[4]) {
  const uint32_t a = w[q >> 1], b = w[q >> 1] >> 10;
  if (q & 1)
    v[0] = mask_pair<2, 8>(a), v[1] = mask_pair<2, 0>(b), v[2] = mask_pair<2, 2>(b), v[3] = mask_pair<2, 4>(b);
  else
    v[0] = mask_pair<2, 0>(a), v[1] = mask_pair<2, 2>(a), v[2] = mask_pair<2, 4>(a), v[3] = mask_pair<2, 6>(a);
}
template <>
__device__ __forceinline__ void unit_quad<3>(const uint32_t (&w)[3], int q, uint32_t (&v)[4]) {
  // words 0, 1, 2 hold codes 0-9, 11-20 and 22-31 whole, from bits 0, 1 and 2: runs of five, two to a register
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = 4 * q + j;
    if (i == 15) {
      v[j] = mask_pair<3, 0>(__byte_perm(__funnelshift_r(w[0], w[1], 30), __funnelshift_r(w[1], w[2], 31), 0x5410));
    } else {
      const uint32_t b = w[1] >> 1, c = w[2] >> 2;
      const uint32_t run = i < 5 ? __byte_perm(w[0], b, 0x5410)
                                 : (i < 10 ? __byte_perm(w[0] >> 15, b >> 15, 0x5410) : __byte_perm(c, c >> 15, 0x5410));
      const int s = i % 5;
      const uint32_t r = s < 3 ? run : run >> 9;
      v[j] = s % 3 == 0 ? mask_pair<3, 0>(r) : (s % 3 == 1 ? mask_pair<3, 3>(r) : mask_pair<3, 6>(r));
    }
  }
}

// (q - zero) 2^p of two codes, exact: q 2^p and zero 2^p are the low mantissa bits of 1024 + ...
__device__ __forceinline__ uint32_t less_zero(uint32_t q, uint32_t zero) {
  q |= 0x64006400u, zero |= 0x64006400u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&q), *reinterpret_cast<const __half2*>(&zero));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------ chained launches
// All launches but the first may start while the one before still runs (programmatic dependent launch): their
// threads wait here, before they touch memory, until it has ended and its writes are visible.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid), cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// ------------------------------------------------------------------ workspace
struct Tile {  // up to 8 NT tokens of one expert: entries [first, first + count) of the pair list
  int32_t expert, first, count;
};
struct Lists {
  int32_t n_tiles;
  int32_t pad[3];
  Tile tiles[kMaxPairs];
  int32_t pairs[kMaxPairs];  // pair = token * top_k + place in the token's choice, grouped by expert
};

// fp16 terms of rows of columns, in the order of Pairs
struct Terms {
  uint16_t* values;   // [term][row][chunk][quad of registers][unit of the chunk][register of the quad]
  float2* chunk;      // [row][chunk]: 2^e, sum of x 2^(-e - 24) over the chunk
  float* unit;        // [row][unit of every chunk]: the same sum over the unit
  int64_t stride;     // values per term
  int chunks;         // 128-column chunks per row
};

struct Layout {
  size_t lists, logits, x_terms, a_terms, acts, products, total;
};
int chunks_of(int64_t cols) { return (int)((cols + 255) / 256 * 2); }  // whole spans of two
size_t terms_bytes(int64_t rows, int64_t cols) {
  return (size_t)rows * chunks_of(cols) * (2 * 256 + sizeof(float2) + 4 * sizeof(float));
}
Layout layout_of(int64_t tokens, int64_t d, int64_t f, int64_t top_k, int64_t experts) {
  Layout l;
  const size_t pairs = (size_t)tokens * top_k;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  l.lists = take(sizeof(Lists));
  l.logits = take((size_t)tokens * experts * 4);
  l.x_terms = take(terms_bytes(tokens, d));
  l.a_terms = take(terms_bytes(pairs, f));
  l.acts = take(pairs * f * 4);
  l.products = take(pairs * d * 4);
  l.total = at;
  return l;
}
Terms terms_at(void* base, int64_t rows, int64_t cols) {
  Terms t;
  t.chunks = chunks_of(cols);
  t.stride = rows * t.chunks * 128;
  t.values = static_cast<uint16_t*>(base);
  t.unit = reinterpret_cast<float*>(t.values + 2 * t.stride);  // a chunk's four start on 16 bytes
  t.chunk = reinterpret_cast<float2*>(t.unit + 4 * rows * t.chunks);
  return t;
}

// ------------------------------------------------------------------ router logits, tokens' layout
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      T lo = reinterpret_cast<const T*>(&w[i])[0], hi = reinterpret_cast<const T*>(&w[i])[1];
      v[2 * i] = to_f32<T>(lo), v[2 * i + 1] = to_f32<T>(hi);
    }
  }
}

// The terms of one row's unit u of 32 columns (zeros past the last unit); the four lanes of a chunk call it
// together.
template <typename T, int BITS, int TERMS>
__device__ __forceinline__ void layout_unit(const T* __restrict__ row, int64_t r, int u, int units, const Terms& out) {
  float v[32];
  float big = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (u < units) load8<T>(row + u * 32 + 8 * q, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[8 * q + k] = x[k];
      const float m = fabsf(x[k]);
      big = fmaxf(big, m < INFINITY ? m : 0.0f);
    }
  }
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
  // 2^(e + 14) <= big < 2^(e + 15)
  const int e = big > 0.0f ? max((int)(__float_as_uint(big) >> 23) - 127 - 14, -126) : 0;
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
  float sum = 0.0f;
  uint32_t out_v[TERMS][16];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] *= down;  // exact
    sum += v[i];
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float scale = 1.0f / (float)(1 << Pairs<BITS>::p(i));
    float x[2] = {v[Pairs<BITS>::lo(i)] * scale, v[Pairs<BITS>::hi(i)] * scale};
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
      uint32_t word = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const __half t = __float2half_rn(x[h]);
        word |= (uint32_t)__half_as_ushort(t) << (16 * h);
        x[h] = fabsf(x[h]) < INFINITY ? x[h] - __half2float(t) : 0.0f;
      }
      out_v[k][i] = word;
    }
  }
#pragma unroll
  for (int k = 0; k < TERMS; ++k) {
    uint4* dst = reinterpret_cast<uint4*>(out.values + k * out.stride + (r * out.chunks + (u >> 2)) * 128) + (u & 3);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      dst[4 * q] = make_uint4(out_v[k][4 * q], out_v[k][4 * q + 1], out_v[k][4 * q + 2], out_v[k][4 * q + 3]);
  }
  constexpr float kCode = 1.0f / 16777216.0f;  // 2^-24, a code's unit
  out.unit[r * out.chunks * 4 + u] = sum * kCode;
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  if ((u & 3) == 0) out.chunk[r * out.chunks + (u >> 2)] = make_float2(__uint_as_float((uint32_t)(e + 127) << 23), sum * kCode);
}

constexpr int kRouterTokens = 8;  // tokens per CTA of the logits

// Logits of one expert for up to 8 tokens, by a CTA of 256 threads: item = token group * experts + expert.
template <typename T>
__device__ __forceinline__ void router_logits(const T* __restrict__ X, const T* __restrict__ R, int tokens, int d,
                                              int experts, int item, float* logits) {
  const int e = item % experts, t0 = item / experts * kRouterTokens;
  const int nt = min(kRouterTokens, tokens - t0);
  float acc[kRouterTokens];
#pragma unroll
  for (int t = 0; t < kRouterTokens; ++t) acc[t] = 0.0f;
  for (int c = threadIdx.x * 8; c < d; c += 256 * 8) {
    float r[8];
    load8<T>(R + (int64_t)e * d + c, r);
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) {
      if (t < nt) {
        float x[8];
        load8<T>(X + (int64_t)(t0 + t) * d + c, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t] = fmaf(x[i], r[i], acc[t]);
      }
    }
  }
  __shared__ float part[8][kRouterTokens];
#pragma unroll
  for (int t = 0; t < kRouterTokens; ++t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][t] = acc[t];
  }
  __syncthreads();
  if ((int)threadIdx.x < nt) {
    float s = 0.0f;
    for (int w = 0; w < 8; ++w) s += part[w][threadIdx.x];
    logits[(int64_t)(t0 + threadIdx.x) * experts + e] = s;
  }
}

// The layout of rows of values, a thread per unit of 32 columns: thread i of them all.
template <typename T, int BITS, int TERMS>
__device__ __forceinline__ void layout_thread(const T* __restrict__ X, int64_t rows, int cols, int64_t i,
                                              const Terms& terms) {
  const int per_row = terms.chunks * 4;
  const int64_t n = rows * per_row;
  const int64_t r = min(i, n - 1) / per_row;  // past the end: the last chunk once more (whole warps shuffle)
  const int u = (int)(i < n ? i - r * per_row : per_row - 4 + (i & 3));
  layout_unit<T, BITS, TERMS>(X + r * cols, r, u, cols >> 5, terms);
}

// CTAs [0, experts * token groups): an item of the logits each.  The others: the tokens' layout.
template <typename T, int BITS, int TERMS>
__global__ void __launch_bounds__(256) moe_router_kernel(const T* __restrict__ X, const T* __restrict__ R, int tokens,
                                                         int d, int experts, int router_blocks,
                                                         float* __restrict__ logits, const Terms terms) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if ((int)blockIdx.x < router_blocks)
    router_logits<T>(X, R, tokens, d, experts, blockIdx.x, logits);
  else
    layout_thread<T, BITS, TERMS>(X, tokens, d, (int64_t)(blockIdx.x - router_blocks) * 256 + threadIdx.x, terms);
}

// the activations' layout
template <int BITS, int TERMS>
__global__ void __launch_bounds__(256) moe_layout_kernel(const float* __restrict__ acts, int64_t rows, int cols,
                                                         const Terms terms) {
  wait_for_previous();
  layout_thread<float, BITS, TERMS>(acts, rows, cols, (int64_t)blockIdx.x * 256 + threadIdx.x, terms);
}

// ------------------------------------------------------------------ top-K and the lists
__device__ __forceinline__ uint32_t ordered(float v) {  // larger float <=> larger integer
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// By one CTA of WARPS warps.  A warp per token chooses its experts (largest logits first, ties to the lowest index) and
// their weights; then a warp per expert collects its pairs in order.
struct Route {
  int tokens, experts, top_k, renormalize, tile_tokens;
  int32_t* ids;
  float* weights;
  Lists* lists;
  int32_t* status;
};
template <int WARPS>
__device__ __forceinline__ void route(const float* logits, const Route& a) {
  __shared__ int32_t id_of[kMaxPairs];
  __shared__ int32_t first_of[kMaxExperts], count_of[kMaxExperts], tile_of[kMaxExperts];
  const int tokens = a.tokens, experts = a.experts, top_k = a.top_k, tile_tokens = a.tile_tokens;
  int32_t* ids = a.ids;
  Lists* lists = a.lists;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = tokens * top_k;
  if (logits != nullptr) {
    for (int t = warp; t < tokens; t += WARPS) {
      constexpr int N = kMaxExperts / 32;
      const int n = (experts + 31) >> 5;  // of them in use
      float l[N];
      uint32_t key[N];
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i >= n) break;
        const int e = lane + 32 * i;
        l[i] = e < experts ? __ldcg(logits + t * experts + e) : -INFINITY;
        key[i] = e < experts ? max(ordered(l[i]), 1u) : 0u;  // 0: not there, or chosen before
        mx = fmaxf(mx, l[i]);
      }
      mx = warp_max(mx);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i >= n) break;
        if (lane + 32 * i < experts) sum += expf(l[i] - mx);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      float mine = 0.0f, chosen = 0.0f;  // lane k keeps the k-th weight
      for (int k = 0; k < top_k; ++k) {
        uint32_t best = 0, at = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (i >= n) break;
          best = max(best, key[i]);
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (i >= n) break;
          if (key[i] == top) at = min(at, (uint32_t)(lane + 32 * i));
        }
        const int e = (int)__reduce_min_sync(0xffffffffu, at);
        float le = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (i >= n) break;
          if (lane + 32 * i == e) le = l[i], key[i] = 0;
        }
        le = __shfl_sync(0xffffffffu, le, e & 31);
        const float w = expf(le - mx) / sum;
        chosen += w;
        if (lane == k) mine = w;
        if (lane == 0) {
          ids[t * top_k + k] = e;
          id_of[t * top_k + k] = e;
        }
      }
      if (lane < top_k) a.weights[t * top_k + lane] = a.renormalize ? mine / chosen : mine;
    }
  } else {
    for (int p = threadIdx.x; p < pairs; p += 32 * WARPS) {
      const int e = ids[p];
      if (e < 0 || e >= experts) report_status(a.status, GPTQ_ERR_ARG, p);
      id_of[p] = e;
    }
  }
  __syncthreads();
  for (int e = warp; e < experts; e += WARPS) {
    int count = 0;
    for (int p = lane; p - lane < pairs; p += 32) count += __popc(__ballot_sync(0xffffffffu, p < pairs && id_of[p] == e));
    if (lane == 0) first_of[e] = count_of[e] = count, tile_of[e] = (count + tile_tokens - 1) / tile_tokens;
  }
  __syncthreads();
  if (warp == 0) {  // exclusive sums over the experts, 32 at a time
    int pair_base = 0, tile_base = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
      const int c = e0 + lane < experts ? first_of[e0 + lane] : 0, n = e0 + lane < experts ? tile_of[e0 + lane] : 0;
      int cs = c, ns = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, cs, o), b = __shfl_up_sync(0xffffffffu, ns, o);
        if (lane >= o) cs += a, ns += b;
      }
      if (e0 + lane < experts) {
        first_of[e0 + lane] = pair_base + cs - c;
        tile_of[e0 + lane] = tile_base + ns - n;
      }
      pair_base += __shfl_sync(0xffffffffu, cs, 31);
      tile_base += __shfl_sync(0xffffffffu, ns, 31);
    }
    if (lane == 0) lists->n_tiles = tile_base;
  }
  __syncthreads();
  for (int e = warp; e < experts; e += WARPS) {
    int at = first_of[e];
    const int count = count_of[e];
    for (int i = lane; i * tile_tokens < count; i += 32)
      lists->tiles[tile_of[e] + i] = {e, at + i * tile_tokens, min(count - i * tile_tokens, tile_tokens)};
    for (int p = lane; p - lane < pairs; p += 32) {
      const bool mine = p < pairs && id_of[p] == e;
      const uint32_t all = __ballot_sync(0xffffffffu, mine);
      if (mine) lists->pairs[at + __popc(all & ((1u << lane) - 1u))] = p;
      at += __popc(all);
    }
  }
}

__global__ void __launch_bounds__(1024) moe_route_kernel(const float* logits, const Route a) {
  wait_for_previous();
  route<32>(logits, a);
}

// Router and choice in one launch, where the logits are at most an item for each CTA of a cluster: when all are there its
// first CTA chooses.  The other clusters: the tokens' layout.  In a graph the two forms take the same (1 token,
// 8 experts, d 4096: 17.4 us the layer with f = 256), and the host has one launch less (5 tokens, 4 experts of 768 x 768
// called from Python: 25.4 -> 22.7 us); with two items a CTA the launch saved is lost again (8 tokens, 16
// experts: 28.8 -> 33.5).
constexpr int kRouteCluster = 8;
template <typename T, int BITS, int TERMS>
__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(256)
    moe_router_route_kernel(const T* __restrict__ X, const T* __restrict__ R, int d, int items, float* logits,
                            const Terms terms, const Route a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x >= kRouteCluster) {
    layout_thread<T, BITS, TERMS>(X, a.tokens, d, (int64_t)(blockIdx.x - kRouteCluster) * 256 + threadIdx.x, terms);
    return;
  }
  if ((int)blockIdx.x < items) router_logits<T>(X, R, a.tokens, d, a.experts, blockIdx.x, logits);
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (blockIdx.x == 0) route<8>(R != nullptr ? logits : nullptr, a);
}

// ------------------------------------------------------------------ products with packed weights
enum { kUpGated = 0, kUpRelu = 1, kDown = 2 };

struct Matrix {
  const uint32_t* words;
  const float* scales;
  const int32_t* zeros;
};

struct ProductArgs {
  Matrix a, b;             // gated: gate and up; else a is the matrix
  int mode, rows, units;   // rows per expert, units of 32 columns per row
  int ng, group_units;     // grids per row, units per grid
  uint32_t grid_magic;     // ceil(2^32 / group_units): u / group_units in the high word, exact for u < 2^16
  int spans;               // of 256 columns, two chunks
  bool wide_rows;          // rows of codes start on 16 bytes
  bool grid_pairs;         // a span's two grids are neighbours and start on 8 bytes
  int row_tiles;           // 32-row (gated: 16-row) tiles of an expert
  int k_warps;             // warps that share a row tile's chunks: 1, 2, 4 or 8
  int cols;                // tokens of a tile at most
  int top_k, pairs;
  Terms terms;             // rows: tokens (up) or pairs (down)
  const Lists* lists;
  float* out;              // [pair][rows]: activations (up) or products (down)
};

constexpr int kProductWarps = 8;
constexpr int kStages = 2;
constexpr float kCodeInverse = 16777216.0f;  // 2^24

constexpr int kCtasPerSm = 2;  // registers (128 a thread) and shared memory are held to it

// Shared memory of one stage, a span of 256 columns: every warp's codes and grids, every group's tokens.
// A row's codes of a span take 128, 96 or 64 bytes; their 16-byte pieces are laid out so that the 8 rows of an
// M tile's half fall into different banks when each lane reads its unit: 3 bits by a row stride of 112 bytes, 4 and 2
// bits by exchanging the halves of every second row, or of every second pair of rows (half_bit).
template <int BITS>
__host__ __device__ constexpr int code_stride() {
  return BITS == 3 ? 112 : 32 * BITS;
}
template <int BITS>
__host__ __device__ constexpr int half_bit(int row) {
  return BITS == 4 ? row & 1 : (BITS == 2 ? row >> 1 & 1 : 0);
}
template <int BITS, int SUB>
__host__ __device__ constexpr int warp_stage_bytes() {
  return 32 * code_stride<BITS>() + 2 * 32 * 2 * SUB * 4;
}
__host__ __device__ inline int token_stage_bytes(int cols, int terms, int sub) {
  return cols * (terms * 512 + 16 + (sub > 1 ? 32 : 0));
}

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool ok = true) {  // zeros where !ok
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(ok ? N : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row tile is 32 weight rows as two M tiles of 16 (consecutive rows, or the same 16 rows of gate and up) of one
// expert, times up to 8 NT of its tokens.  The CTA's 8 warps are k_warps groups: a group's warps take
// neighbouring row tiles and the same spans (every k_warps-th), so they share the tokens' terms; the groups'
// sums are added in order through shared memory at the end.  Codes, grids, and tokens' terms arrive in a ring
// of stages by asynchronous copies a span of two chunks ahead, across the borders of work items, without holding
// registers: with the next chunk in registers the same products took 2.3 us a chunk and warp, most of it waiting.
// In a chunk the four lanes of a row take a unit of 32 codes each.  After each chunk the sums over its 128
// columns are scaled into fp32 sums.
// SUB: scales change inside a chunk (groups of 32 or 64); each quarter then has accumulators of its own and
// sees the other quarters' tokens as zeros.
// PRECISE: zero points off the codes (see the top), else through the tokens' sums.
template <int BITS, int TERMS, int NT, int SUB, bool PRECISE>
__global__ void __launch_bounds__(kProductWarps * 32, kCtasPerSm) moe_product_kernel(const ProductArgs a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float sums[kProductWarps][32][8 * NT + 1];
  __shared__ uint16_t pair_of[kMaxPairs], row_of[kMaxPairs];  // pairs by expert; their rows of the terms
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int groups = kProductWarps / a.k_warps;                  // row tiles of an item
  const int kw = warp / groups, rg = warp - kw * groups;
  const int per_tile = (a.row_tiles + groups - 1) / groups;
  const bool gated = a.mode == kUpGated;
  const int tile_rows = gated ? 16 : 32;
  const int64_t row_words = (int64_t)a.units * BITS;
  wait_for_previous();
  if ((int)blockIdx.x >= a.lists->n_tiles * per_tile) return;
  for (int i = threadIdx.x; i < a.pairs; i += kProductWarps * 32) {
    const int p = a.lists->pairs[i];
    pair_of[i] = (uint16_t)p;
    row_of[i] = (uint16_t)(a.mode == kDown ? p : p / a.top_k);
  }
  __syncthreads();

  constexpr int WS = warp_stage_bytes<BITS, SUB>();
  constexpr int RS = code_stride<BITS>(), HB = 16 * BITS;  // bytes of a row; of a row's half of a span
  const int ts = token_stage_bytes(a.cols, TERMS, SUB);
  const int stage_bytes = kProductWarps * WS + a.k_warps * ts;
  const uint32_t ring0 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t ring_end = kStages * stage_bytes;
  const int my_codes = warp * WS, my_tokens = kProductWarps * WS + kw * ts;
  const int steps = a.spans > kw ? (a.spans - kw + a.k_warps - 1) / a.k_warps : 0;  // this group's spans

  // ---- the copies: span after span of item after item
  const int gt = rg * 32 + lane;  // this thread among its group's
  // an item is row tiles in_rt .. of list tile in_tile; the next one lies gridDim.x items further on
  const int hop_tile = (int)gridDim.x / per_tile, hop_rt = (int)gridDim.x % per_tile;
  auto hop = [&](int& tile, int& rt) {
    tile += hop_tile, rt += hop_rt;
    if (rt >= per_tile) rt -= per_tile, ++tile;
  };
  int in_tile = (int)blockIdx.x / per_tile, in_rt = (int)blockIdx.x % per_tile, in_c = kw;
  const int n_tiles = a.lists->n_tiles;
  uint32_t in_stage = 0;
  int in_first = 0, in_count = 0;
  const uint32_t *words0 = nullptr, *words1 = nullptr;  // span in_c of the M tiles' first rows
  const float* scales = nullptr;       // row `lane` of the tile
  const int32_t* zeros = nullptr;
  const char* term0 = reinterpret_cast<const char*>(a.terms.values) + lane * 16;
  const char* term1 = term0 + 2 * a.terms.stride;
  // This lane's 16-byte pieces of an M tile's codes: piece p = lane + 32 i is piece p % PP of row p / PP.  From
  // the tile's first row to them, in words and in bytes of the stage:
  constexpr int PP = 2 * BITS, NI = 16 * PP / 32;
  int src_of[NI], dst_of[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int row = (lane + 32 * i) / PP, at = (lane + 32 * i) % PP;
    src_of[i] = row * (int)row_words + at * 4;
    dst_of[i] = row * RS + (at ^ (half_bit<BITS>(row) * BITS)) * 16;
  }
  const uint32_t grid_magic = a.grid_magic;
  auto grid_of = [&](int u) {  // u / group_units
    return SUB > 1 ? u >> (a.group_units - 1) : (int)__umulhi((uint32_t)u, grid_magic);
  };
  auto begin_item = [&]() {
    if (in_tile >= n_tiles) return;
    const Tile tile = a.lists->tiles[in_tile];
    in_first = tile.first, in_count = tile.count;
    const int64_t r = (int64_t)tile.expert * a.rows + min(in_rt * groups + rg, a.row_tiles - 1) * tile_rows;
    words0 = a.a.words + r * row_words + kw * (8 * BITS);
    words1 = gated ? a.b.words + r * row_words + kw * (8 * BITS) : words0 + 16 * row_words;
    const int64_t lane_row = (r + (gated ? lane & 15 : lane)) * a.ng;
    scales = (gated && lane >= 16 ? a.b.scales : a.a.scales) + lane_row;
    zeros = (gated && lane >= 16 ? a.b.zeros : a.a.zeros) + lane_row;
  };
  auto issue = [&]() {
    if (in_tile < n_tiles && steps > 0) {
      const uint32_t stage = ring0 + in_stage, codes = stage + my_codes;
      const int c = in_c;
      const int left = (int)row_words - c * (8 * BITS);  // words of a row from here on
      if (BITS == 4 || a.wide_rows) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const bool ok = left >= 8 * BITS || (lane + 32 * i) % PP * 4 < left;
          copy_async<16>(codes + dst_of[i], words0 + (ok ? src_of[i] : 0), ok);
          copy_async<16>(codes + 16 * RS + dst_of[i], words1 + (ok ? src_of[i] : 0), ok);
        }
      } else {  // rows on any 4 bytes: row `lane`, word by word
        const uint32_t* src = (lane < 16 ? words0 : words1) + (lane & 15) * row_words;
#pragma unroll 1
        for (int p = 0; p < 8 * BITS; ++p) {
          const bool ok = p < left;
          copy_async<4>(codes + lane * RS + ((p >> 2) ^ (half_bit<BITS>(lane) * BITS)) * 16 + (p & 3) * 4, ok ? src + p : src, ok);
        }
      }
      const uint32_t grids = codes + 32 * RS + lane * (2 * SUB * 4);  // [row][chunk, quarter] scales, then zeros
      if (SUB == 1 && a.grid_pairs) {
        copy_async<8>(grids, scales + 2 * c);
        copy_async<8>(grids + 32 * 2 * 4, zeros + 2 * c);
      } else {
#pragma unroll
        for (int s = 0; s < 2 * SUB; ++s) {
          const int grid = grid_of(min(8 * c + (SUB == 1 ? 4 * s : s), a.units - 1));
          copy_async<4>(grids + s * 4, scales + grid);
          copy_async<4>(grids + (32 * 2 * SUB + s) * 4, zeros + grid);
        }
      }
      // the group's warps share its tokens: 32 pieces per token and term, odd tokens' neighbouring quads exchanged
      // so that two tokens' pieces of one quad lie in different banks.  (Offsets from a term's start fit 32 bits: at
      // most 1024 rows of 8192 chunks of 256 bytes.)
      const uint32_t tokens = stage + my_tokens;
      for (int i = rg; i < in_count * TERMS; i += groups) {
        const int j = TERMS == 1 ? i : i >> 1;
        const uint32_t at = (uint32_t)row_of[in_first + j] * (uint32_t)a.terms.chunks + 2u * (uint32_t)c;
        copy_async<16>(tokens + i * 512 + (lane ^ 4 * (j & 1)) * 16, (TERMS > 1 && (i & 1) ? term1 : term0) + (at << 8));
      }
      if (gt < in_count) {  // at most 16 tokens: the group's first warp
        const uint32_t stats = tokens + a.cols * (TERMS * 512);
        const uint32_t at = (uint32_t)row_of[in_first + gt] * (uint32_t)a.terms.chunks + 2u * (uint32_t)c;
        copy_async<16>(stats + gt * 16, a.terms.chunk + at);
        if constexpr (SUB > 1 && !PRECISE) {
          copy_async<16>(stats + a.cols * 16 + gt * 32, a.terms.unit + at * 4);
          copy_async<16>(stats + a.cols * 16 + gt * 32 + 16, a.terms.unit + at * 4 + 4);
        }
      }
      in_c += a.k_warps;
      words0 += a.k_warps * (8 * BITS), words1 += a.k_warps * (8 * BITS);
      if (in_c >= a.spans) {
        in_c = kw;
        hop(in_tile, in_rt);
        begin_item();
      }
    }
    copies_commit();
    in_stage += stage_bytes;
    if (in_stage == ring_end) in_stage = 0;
  };
  begin_item();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue();

  uint32_t out_stage = 0;
  int at_tile = -1, first = 0, count = 0;
  int tok[NT], col[NT][2];
  int tile = (int)blockIdx.x / per_tile, rt0 = (int)blockIdx.x % per_tile;
  for (; tile < n_tiles; hop(tile, rt0)) {
    if (tile != at_tile) {
      at_tile = tile;
      first = a.lists->tiles[tile].first, count = a.lists->tiles[tile].count;
      // Columns past the tile's last token repeat it (nobody reads them).  This lane's column of B is entry g of every
      // 8 (quad 0's piece; quad q's is that with q exchanged into its place), its columns of the sums are
      // entries 2 t and 2 t + 1.
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int j = min(8 * n + g, count - 1);
        tok[n] = j * (TERMS * 512) + ((t ^ 4 * (j & 1)) << 4);
        col[n][0] = min(8 * n + 2 * t, count - 1), col[n][1] = min(8 * n + 2 * t + 1, count - 1);
      }
    }
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
    for (int step = 0; step < steps; ++step) {
      copies_wait<kStages - 2>();
      // the group's copies of this stage have landed and its reads of the one before are done
      if (groups == 1)
        __syncwarp();
      else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + kw), "r"(groups * 32) : "memory");
      issue();
      const uint8_t* stage = ring + out_stage;
      out_stage += stage_bytes;
      if (out_stage == ring_end) out_stage = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // the span's chunks
        const uint8_t* codes = stage + my_codes;
        uint32_t w[4][BITS];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t* p = reinterpret_cast<const uint32_t*>(codes + (8 * i + g) * RS + (h ^ half_bit<BITS>(g)) * HB + t * (4 * BITS));
          if constexpr (BITS == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
          } else if constexpr (BITS == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[i][0] = v.x, w[i][1] = v.y;
          } else {
#pragma unroll
            for (int k = 0; k < BITS; ++k) w[i][k] = p[k];
          }
        }
        // row g + 8 i: 16 SUB i further
        const float* sc = reinterpret_cast<const float*>(codes + 32 * RS) + g * (2 * SUB) + h * SUB;
        const int32_t* zr = reinterpret_cast<const int32_t*>(codes + 32 * RS) + 32 * 2 * SUB + g * (2 * SUB) + h * SUB;
        const uint8_t* tokens = stage + my_tokens + h * 256;
        const float2* stats = reinterpret_cast<const float2*>(stage + my_tokens + a.cols * (TERMS * 512)) + h;
        const float* unit_sums = reinterpret_cast<const float*>(stage + my_tokens + a.cols * (TERMS * 512 + 16)) + h * 4;
        // the accumulators start at -zero sum x (PRECISE: at zero); row g of an M tile is in values 0 and 1, row g + 8
        // in 2 and 3
        float sum[NT][SUB][2][4];
        float2 st[NT][2];
        uint32_t zp[4];  // PRECISE: this lane's unit's zeros, in both halves
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n == 0 || 8 * n < count) st[n][0] = stats[2 * col[n][0]], st[n][1] = stats[2 * col[n][1]];
#pragma unroll
        for (int i = 0; i < 4; ++i) zp[i] = PRECISE ? ((uint32_t)zr[16 * SUB * i + (SUB == 1 ? 0 : t)] & ((1u << BITS) - 1u)) * 0x10001u : 0u;
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          float z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = PRECISE ? 0.0f : -(float)zr[16 * SUB * i + s];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n > 0 && 8 * n >= count) break;
            const float x0 = PRECISE ? 0.0f : (SUB == 1 ? st[n][0].y : unit_sums[8 * col[n][0] + s]);
            const float x1 = PRECISE ? 0.0f : (SUB == 1 ? st[n][1].y : unit_sums[8 * col[n][1] + s]);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              sum[n][s][m][0] = PRECISE ? 0.0f : z[2 * m] * x0, sum[n][s][m][1] = PRECISE ? 0.0f : z[2 * m] * x1;
              sum[n][s][m][2] = PRECISE ? 0.0f : z[2 * m + 1] * x0, sum[n][s][m][3] = PRECISE ? 0.0f : z[2 * m + 1] * x1;
            }
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // registers 4 q .. 4 q + 3 of the units: 32 of the chunk's columns
          uint32_t v[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            unit_quad<BITS>(w[i], q, v[i]);
            if constexpr (PRECISE) {
#pragma unroll
              for (int j = 0; j < 4; ++j) v[i][j] = less_zero(v[i][j], zp[i] << Pairs<BITS>::p(4 * q + j));
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n > 0 && 8 * n >= count) break;
#pragma unroll
            for (int k = TERMS - 1; k >= 0; --k) {
              const uint4 x = *reinterpret_cast<const uint4*>(tokens + (tok[n] ^ (q & 1) << 6) + (q >> 1) * 128 + k * 512);
#pragma unroll
              for (int m = 0; m < 2; ++m) {
#pragma unroll
                for (int s = 0; s < SUB; ++s) {
                  const bool mine = SUB == 1 || t == s;
                  mma_f16(sum[n][s][m], v[2 * m][0], v[2 * m + 1][0], v[2 * m][1], v[2 * m + 1][1], mine ? x.x : 0u,
                          mine ? x.y : 0u);
                  mma_f16(sum[n][s][m], v[2 * m][2], v[2 * m + 1][2], v[2 * m][3], v[2 * m + 1][3], mine ? x.z : 0u,
                          mine ? x.w : 0u);
                }
              }
            }
          }
        }
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          float ss[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) ss[i] = sc[16 * SUB * i + s];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n > 0 && 8 * n >= count) break;
            const float e0 = st[n][0].x, e1 = st[n][1].x;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              acc[m][n][0] = fmaf(ss[2 * m] * e0, sum[n][s][m][0], acc[m][n][0]);
              acc[m][n][1] = fmaf(ss[2 * m] * e1, sum[n][s][m][1], acc[m][n][1]);
              acc[m][n][2] = fmaf(ss[2 * m + 1] * e0, sum[n][s][m][2], acc[m][n][2]);
              acc[m][n][3] = fmaf(ss[2 * m + 1] * e1, sum[n][s][m][3], acc[m][n][3]);
            }
          }
        }
      }
    }
    __syncthreads();  // the last item's sums have been read
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float* lo = &sums[warp][16 * m + g][8 * n + 2 * t];
        float* hi = &sums[warp][16 * m + g + 8][8 * n + 2 * t];
        lo[0] = acc[m][n][0], lo[1] = acc[m][n][1], hi[0] = acc[m][n][2], hi[1] = acc[m][n][3];
      }
    __syncthreads();
    const int out_rows = groups * tile_rows;  // powers of two
    for (int i = threadIdx.x; i < out_rows * count; i += kProductWarps * 32) {
      const int r = i & (tile_rows - 1), j = (i & (out_rows - 1)) >> (gated ? 4 : 5), n = i >> (31 - __clz(out_rows));
      const int rt = rt0 * groups + j;
      if (rt >= a.row_tiles) continue;
      float v = 0.0f, up = 0.0f;
      for (int w = j; w < kProductWarps; w += groups) {
        v += sums[w][r][n];
        if (gated) up += sums[w][16 + r][n];
      }
      if (!PRECISE) v *= kCodeInverse, up *= kCodeInverse;  // codes were taken as q 2^-24
      if (gated)
        v = v / (1.0f + expf(-v)) * up;
      else if (a.mode == kUpRelu)
        v = v < 0.0f ? 0.0f : v;  // NaN stays
      a.out[(int64_t)pair_of[first + n] * a.rows + rt * tile_rows + r] = v;
    }
  }
  copies_wait<0>();
}

// ------------------------------------------------------------------ weighted sum
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename TY>
__global__ void __launch_bounds__(256) moe_combine_kernel(const float* __restrict__ products,
                                                          const int32_t* __restrict__ ids,
                                                          const float* __restrict__ weights, int tokens, int d,
                                                          int top_k, int experts, TY* __restrict__ Y) {
  wait_for_previous();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)tokens * d) return;
  const int t = (int)(i / d), c = (int)(i % d);
  float s = 0.0f;
  for (int k = 0; k < top_k; ++k) {
    const int p = t * top_k + k;
    const int e = ids[p];
    if (e >= 0 && e < experts) s = fmaf(weights[p], products[(int64_t)p * d + c], s);
  }
  Y[i] = from_f32<TY>(s);
}

// ------------------------------------------------------------------ launches
// Groups per CTA (warps per row tile): the fewest span steps along the longest chain of work items, an item's own
// start and end counted as one, among those whose stages leave room for the SM's other CTAs.
template <int BITS, int TERMS, int NT, int SUB>
int choose_k_warps(const ProductArgs& a, int tiles, int slots, int* smem) {
  // an SM's 227 KB, less 1 KB and the static arrays of each CTA
  constexpr int kRoom = 227 * 1024 / kCtasPerSm - 1024 - kProductWarps * 32 * (8 * NT + 1) * 4 - 4 * kMaxPairs;
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int kw = 8; kw >= 1; kw /= 2) {
    const int bytes = kStages * (kProductWarps * warp_stage_bytes<BITS, SUB>() + kw * token_stage_bytes(a.cols, TERMS, SUB));
    const int groups = kProductWarps / kw;
    const int64_t items = (int64_t)tiles * ((a.row_tiles + groups - 1) / groups);
    // few groups read short runs of many rows at once, and DRAM answers more slowly: one token on 4096 x 11008
    // experts took 52, 53, 88 and 122 us with 8, 4, 2 and 1
    const int64_t cost = (items + slots - 1) / slots * ((a.spans + kw - 1) / kw + 1) * (kw >= 4 ? 8 : (kw == 2 ? 13 : 18));
    if (best_cost == INT64_MAX ? bytes <= kRoom || kw == 1 : bytes <= kRoom && cost < best_cost)
      best = kw, best_cost = cost, *smem = bytes;
  }
  return best;
}

template <int BITS, int TERMS, int NT, int SUB, bool PRECISE>
gptq_status launch_product_form(ProductArgs a, int tiles, int sms, cudaStream_t s) {
  const int slots = kCtasPerSm * sms;
  int smem = 0;
  a.wide_rows = a.units * BITS % 4 == 0;
  auto pairs_of = [&](const Matrix& w) { return aligned(w.scales, 8) && aligned(w.zeros, 8); };
  a.grid_pairs = a.group_units == 4 && a.ng % 2 == 0 && pairs_of(a.a) && (a.mode != kUpGated || pairs_of(a.b));
  a.grid_magic = (uint32_t)(((1ull << 32) + a.group_units - 1) / a.group_units);  // not used for group_units 1
  a.k_warps = choose_k_warps<BITS, TERMS, NT, SUB>(a, tiles, slots, &smem);
  const int groups = kProductWarps / a.k_warps;
  const int64_t items = (int64_t)tiles * ((a.row_tiles + groups - 1) / groups);
  auto kernel = moe_product_kernel<BITS, TERMS, NT, SUB, PRECISE>;
  GPTQ_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  GPTQ_CUDA_TRY(launch_chained(kernel, (unsigned)std::min<int64_t>(items, slots), kProductWarps * 32, smem, s, a));
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <int BITS, int TERMS, bool PRECISE>
gptq_status launch_product_typed(const ProductArgs& a, int nt, bool sub, int tiles, int sms, cudaStream_t s) {
  if (sub) return launch_product_form<BITS, TERMS, 1, 4, PRECISE>(a, tiles, sms, s);
  return nt == 1 ? launch_product_form<BITS, TERMS, 1, 1, PRECISE>(a, tiles, sms, s)
                 : launch_product_form<BITS, TERMS, 2, 1, PRECISE>(a, tiles, sms, s);
}

template <int BITS>
gptq_status launch_product(bool two_terms, bool precise, const ProductArgs& a, int nt, bool sub, int tiles, int sms,
                           cudaStream_t s) {
  if (precise)
    return two_terms ? launch_product_typed<BITS, 2, true>(a, nt, sub, tiles, sms, s)
                     : launch_product_typed<BITS, 1, true>(a, nt, sub, tiles, sms, s);
  return two_terms ? launch_product_typed<BITS, 2, false>(a, nt, sub, tiles, sms, s)
                   : launch_product_typed<BITS, 1, false>(a, nt, sub, tiles, sms, s);
}

template <typename T, int BITS, int TERMS>
gptq_status launch_router(const MoeArgs& m, float* logits, const Terms& terms, const Route& r, cudaStream_t s) {
  const int tokens = (int)m.tokens, d = (int)m.d;
  const T *X = static_cast<const T*>(m.X), *R = static_cast<const T*>(m.router);
  const int items = m.experts * ((tokens + kRouterTokens - 1) / kRouterTokens);
  const int layout_blocks = (int)(((int64_t)tokens * terms.chunks * 4 + 255) / 256);
  if (items <= kRouteCluster) {
    const int blocks = kRouteCluster + (layout_blocks + kRouteCluster - 1) / kRouteCluster * kRouteCluster;
    moe_router_route_kernel<T, BITS, TERMS><<<blocks, 256, 0, s>>>(X, R, d, R ? items : 0, logits, terms, r);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
  }
  const int router_blocks = R ? items : 0;
  moe_router_kernel<T, BITS, TERMS><<<router_blocks + layout_blocks, 256, 0, s>>>(X, R, tokens, d, m.experts,
                                                                                  router_blocks, logits, terms);
  GPTQ_LAUNCH_CHECK();
  GPTQ_CUDA_TRY(launch_chained(moe_route_kernel, 1, 1024, 0, s, R ? logits : nullptr, r));
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <int BITS>
gptq_status moe_typed(const MoeArgs& m, cudaStream_t s) {
  const Layout l = layout_of(m.tokens, m.d, m.f, m.top_k, m.experts);
  char* ws = static_cast<char*>(m.workspace);
  Lists* lists = reinterpret_cast<Lists*>(ws + l.lists);
  float* logits = reinterpret_cast<float*>(ws + l.logits);
  float* acts = reinterpret_cast<float*>(ws + l.acts);
  float* products = reinterpret_cast<float*>(ws + l.products);
  int dev = 0, sms = 0;
  GPTQ_CUDA_TRY(cudaGetDevice(&dev));
  GPTQ_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  const int tokens = (int)m.tokens, d = (int)m.d, f = (int)m.f;
  const int pairs = tokens * m.top_k;
  const Terms x_terms = terms_at(ws + l.x_terms, tokens, d), a_terms = terms_at(ws + l.a_terms, pairs, f);
  const bool x_wide = m.x_dtype == GPTQ_FP32, a_wide = m.y_dtype != GPTQ_BF16, precise = m.y_dtype == GPTQ_FP32;
  // An expert's list goes 8 tokens at a time, or 16 where lists are long (more than 12 on average), so that the
  // codes are taken apart once for two N tiles; 16 tokens' terms leave fewer groups room, so for short lists they
  // only cost (32 tokens, 6 of 32 experts each: 214 us with 16 at a time, 173 with 8).  Scales that change inside
  // a chunk need the registers of the second N tile.
  const bool sub = m.group_size == 32 || m.group_size == 64;
  const int nt = pairs <= 12 * m.experts || sub ? 1 : 2;
  const int tile_tokens = 8 * nt;
  const int tiles = std::min(pairs, std::min(m.experts, pairs) + pairs / tile_tokens);  // at most
  const Route r = {tokens, m.experts, m.top_k, m.renormalize, tile_tokens, m.ids, m.weights, lists, m.status};
  gptq_status st;
  switch (m.x_dtype) {
    case GPTQ_BF16: st = launch_router<__nv_bfloat16, BITS, 1>(m, logits, x_terms, r, s); break;
    case GPTQ_FP16: st = launch_router<__half, BITS, 1>(m, logits, x_terms, r, s); break;
    default: st = launch_router<float, BITS, 2>(m, logits, x_terms, r, s); break;
  }
  if (st != GPTQ_OK) return st;
  ProductArgs a = {};
  a.mode = m.gated ? kUpGated : kUpRelu;
  auto matrix = [](const MoePacked& p) {
    return Matrix{reinterpret_cast<const uint32_t*>(p.packed), p.scales, p.zeros};
  };
  a.a = matrix(m.gated ? m.gate : m.up);
  a.b = matrix(m.up);
  a.rows = f, a.units = d / 32;
  a.ng = m.group_size ? d / m.group_size : 1;
  a.group_units = m.group_size ? m.group_size / 32 : a.units;
  a.spans = x_terms.chunks / 2, a.row_tiles = m.gated ? f / 16 : f / 32;
  a.top_k = m.top_k, a.pairs = pairs;
  a.cols = std::min(tile_tokens, m.router ? tokens : pairs);
  a.terms = x_terms;
  a.lists = lists;
  a.out = acts;
  st = launch_product<BITS>(x_wide, precise, a, nt, sub, tiles, sms, s);
  if (st != GPTQ_OK) return st;
  const unsigned layout_blocks = (unsigned)(((int64_t)pairs * a_terms.chunks * 4 + 255) / 256);
  if (a_wide)
    GPTQ_CUDA_TRY(launch_chained(moe_layout_kernel<BITS, 2>, layout_blocks, 256, 0, s, acts, pairs, f, a_terms));
  else
    GPTQ_CUDA_TRY(launch_chained(moe_layout_kernel<BITS, 1>, layout_blocks, 256, 0, s, acts, pairs, f, a_terms));
  GPTQ_LAUNCH_CHECK();
  a.mode = kDown;
  a.a = matrix(m.down);
  a.rows = d, a.units = f / 32;
  a.ng = m.group_size ? f / m.group_size : 1;
  a.group_units = m.group_size ? m.group_size / 32 : a.units;
  a.spans = a_terms.chunks / 2, a.row_tiles = d / 32;
  a.terms = a_terms;
  a.out = products;
  st = launch_product<BITS>(a_wide, precise, a, nt, sub, tiles, sms, s);
  if (st != GPTQ_OK) return st;
  const unsigned blocks = (unsigned)(((int64_t)tokens * d + 255) / 256);
  switch (m.y_dtype) {
    case GPTQ_BF16: GPTQ_CUDA_TRY(launch_chained(moe_combine_kernel<__nv_bfloat16>, blocks, 256, 0, s, products, m.ids, m.weights, tokens, d, m.top_k, m.experts, static_cast<__nv_bfloat16*>(m.Y))); break;
    case GPTQ_FP16: GPTQ_CUDA_TRY(launch_chained(moe_combine_kernel<__half>, blocks, 256, 0, s, products, m.ids, m.weights, tokens, d, m.top_k, m.experts, static_cast<__half*>(m.Y))); break;
    default: GPTQ_CUDA_TRY(launch_chained(moe_combine_kernel<float>, blocks, 256, 0, s, products, m.ids, m.weights, tokens, d, m.top_k, m.experts, static_cast<float*>(m.Y))); break;
  }
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace

size_t moe_workspace(int64_t tokens, int64_t d, int64_t f, int64_t experts, int64_t top_k) {
  return layout_of(tokens, d, f, top_k, experts).total;
}

gptq_status moe_launch(const MoeArgs& m, int32_t bits, cudaStream_t stream) {
  switch (bits) {
    case 2: return moe_typed<2>(m, stream);
    case 3: return moe_typed<3>(m, stream);
    default: return moe_typed<4>(m, stream);
  }
}

}  // namespace gptq
