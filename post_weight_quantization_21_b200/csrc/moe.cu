// A mixture-of-experts layer for a few tokens over packed weights: router, the chosen experts' gate / up
// products, the activation, the down product and the weighted sum.
//   l = x R^T,  p = softmax(l),  e_1 .. e_K = the K largest p,  w_i = p[e_i] (over their sum when renormalised)
//   y = sum_i w_i D_{e_i} a_i,   a_i = silu(G_{e_i} x) * (U_{e_i} x)  or  relu(U_{e_i} x)
// with every matrix What[r, j] = scale[r, g] (q[r, j] - zero[r, g]) read as packed codes.
//
// The bytes of the chosen experts' codes are the floor, so the work to keep below HBM's time is taking the
// codes apart.  A code is masked together with the exponent of 128 into a bf16 mantissa: 128 + q 2^p is
// exact there for q 2^p < 128, and so is the difference with 128 + zero 2^p, (q - zero) 2^p.  Two codes
// per register, one mask and one subtraction per pair, and the pair is a ready fragment of
// mma.m16n8k16 (weights on the M side, up to 8 tokens on the N side): a product of M = 8 tokens is no
// tcgen05 shape, and the tensor pipe has time to spare here.  The order of the columns in a sum is free,
// so the pairs are the codes that lie 16 bits apart (see Pairs) and the tokens' values are laid out to
// match, multiplied by 2^-p.
//
// Tokens are split into bf16 terms that add up to the value exactly: one for bf16, two for fp16, three for
// fp32; the intermediate a_i, kept in fp32, into three, or two when the result has 16 bits (an error of
// 2^-17 beside the result's own 2^-9 or 2^-12).  Every product is then exact in the tensor core, sums
// run there over 128 columns (truncated at 2^-24 or so of the partial sum) and in fp32 beyond.
//
// Launches: router logits and the tokens' layout; top-K and the lists of tokens per expert; the up product
// with the activation; the down product; the weighted sum in the order of the choice.  No atomics: results
// are deterministic.
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
// pair(i) = (column in the low half, column in the high half) of the i-th register of a unit, both masked at
// bit p(i) of their half; the inverse gives a column's register and half.
template <int BITS>
struct Pairs;
template <>
struct Pairs<4> {  // register 4 w + s: word w shifted by 4 s
  __host__ __device__ static constexpr int lo(int i) { return 8 * (i / 4) + i % 4; }
  __host__ __device__ static constexpr int hi(int i) { return lo(i) + 4; }
  __host__ __device__ static constexpr int p(int) { return 0; }
  __host__ __device__ static constexpr int reg(int j) { return 4 * (j / 8) + j % 4; }
  __host__ __device__ static constexpr int half(int j) { return j % 8 / 4; }
};
template <>
struct Pairs<2> {  // register 8 w + s: word w shifted by 6 (s / 3), three codes of a half per shift
  __host__ __device__ static constexpr int lo(int i) { return 16 * (i / 8) + i % 8; }
  __host__ __device__ static constexpr int hi(int i) { return lo(i) + 8; }
  __host__ __device__ static constexpr int p(int i) { return 2 * (i % 8 % 3); }
  __host__ __device__ static constexpr int reg(int j) { return 8 * (j / 16) + j % 8; }
  __host__ __device__ static constexpr int half(int j) { return j % 16 / 8; }
};
template <>
struct Pairs<3> {  // registers 5 b + s: runs of five codes side by side; register 15: the two codes across words
  __host__ __device__ static constexpr int lo(int i) { return i == 15 ? 10 : (i < 5 ? i : (i < 10 ? i : i + 12)); }
  __host__ __device__ static constexpr int hi(int i) { return i == 15 ? 21 : (i < 10 ? i + 11 : i + 17); }
  __host__ __device__ static constexpr int p(int i) { return i == 15 ? 0 : 3 * (i % 5 & 1); }
  __host__ __device__ static constexpr int reg(int j) {
    return j == 10 || j == 21 ? 15 : (j < 10 ? j : (j < 21 ? j - 11 : 10 + (j - 22) % 5));
  }
  __host__ __device__ static constexpr int half(int j) { return j < 11 ? 0 : (j < 22 ? 1 : (j - 22) / 5); }
};
template <int BITS>
__host__ __device__ constexpr bool pairs_ok() {
  for (int i = 0; i < 16; ++i) {
    const int l = Pairs<BITS>::lo(i), h = Pairs<BITS>::hi(i);
    if (Pairs<BITS>::reg(l) != i || Pairs<BITS>::half(l) != 0) return false;
    if (Pairs<BITS>::reg(h) != i || Pairs<BITS>::half(h) != 1) return false;
    if ((((1 << BITS) - 1) << Pairs<BITS>::p(i)) >= 128) return false;
  }
  return true;
}
static_assert(pairs_ok<2>() && pairs_ok<3>() && pairs_ok<4>(), "column order");

constexpr uint32_t kMagic = 0x43004300u;  // 128 in both halves

// (v & (mask << p)) | magic for both halves
template <int BITS, int P>
__device__ __forceinline__ uint32_t mask_pair(uint32_t v) {
  constexpr uint32_t m = ((1u << BITS) - 1u) << P;
  return (v & (m | (m << 16))) | kMagic;
}

// the 16 registers (128 + q 2^p) of a unit
template <int BITS>
__device__ __forceinline__ void unit_pairs(const uint32_t (&w)[BITS], uint32_t (&v)[16]);
template <>
__device__ __forceinline__ void unit_pairs<4>(const uint32_t (&w)[4], uint32_t (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = mask_pair<4, 0>(w[i / 4] >> (4 * (i % 4)));
}
template <>
__device__ __forceinline__ void unit_pairs<2>(const uint32_t (&w)[2], uint32_t (&v)[16]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t a = w[k], b = w[k] >> 6, c = w[k] >> 12;
    v[8 * k + 0] = mask_pair<2, 0>(a), v[8 * k + 1] = mask_pair<2, 2>(a), v[8 * k + 2] = mask_pair<2, 4>(a);
    v[8 * k + 3] = mask_pair<2, 0>(b), v[8 * k + 4] = mask_pair<2, 2>(b), v[8 * k + 5] = mask_pair<2, 4>(b);
    v[8 * k + 6] = mask_pair<2, 0>(c), v[8 * k + 7] = mask_pair<2, 2>(c);
  }
}
template <>
__device__ __forceinline__ void unit_pairs<3>(const uint32_t (&w)[3], uint32_t (&v)[16]) {
  // words 0, 1, 2 hold codes 0-9, 11-20 and 22-31 whole, from bits 0, 1 and 2
  const uint32_t b = w[1] >> 1, c = w[2] >> 2;
  const uint32_t run[3] = {__byte_perm(w[0], b, 0x5410), __byte_perm(w[0] >> 15, b >> 15, 0x5410),
                           __byte_perm(c, c >> 15, 0x5410)};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const uint32_t s6 = run[k] >> 6, s12 = run[k] >> 12;
    v[5 * k + 0] = mask_pair<3, 0>(run[k]), v[5 * k + 1] = mask_pair<3, 3>(run[k]);
    v[5 * k + 2] = mask_pair<3, 0>(s6), v[5 * k + 3] = mask_pair<3, 3>(s6);
    v[5 * k + 4] = mask_pair<3, 0>(s12);
  }
  v[15] = mask_pair<3, 0>(
      __byte_perm(__funnelshift_r(w[0], w[1], 30), __funnelshift_r(w[1], w[2], 31), 0x5410));
}

// 128 + zero 2^p in both halves (zero 2^p < 128 for zeros of the grid; others only use their low bits)
template <int BITS>
__device__ __forceinline__ uint32_t zero_pair(int32_t z, int p) {
  const uint32_t h = 0x4300u | (((uint32_t)z << p) & 0x7Fu);
  return h | (h << 16);
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------ bf16 terms
// v as the sum of `terms` bf16 values, each the nearest to what the ones before leave; a value that is not
// finite is its own first term.
template <int TERMS>
__device__ __forceinline__ void split_bf16(float v, uint16_t (&t)[TERMS]) {
  const bool finite = (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    __nv_bfloat16 h = __float2bfloat16_rn(v);
    // the largest fp32 values round up to infinity: take the largest bf16 and leave the rest to the next term
    if (finite && (__bfloat16_as_ushort(h) & 0x7FFFu) == 0x7F80u && TERMS > 1)
      h = __ushort_as_bfloat16((__bfloat16_as_ushort(h) & 0x8000u) | 0x7F7Fu);
    t[i] = __bfloat16_as_ushort(h);
    v = finite ? v - __bfloat162float(h) : 0.0f;
  }
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

struct Layout {
  size_t lists, logits, x_terms, a_terms, products, total;
  int chunks_d, chunks_f;  // 128-column chunks of a token's and of an intermediate row
};
Layout layout_of(int64_t tokens, int64_t d, int64_t f, int64_t experts, int64_t top_k) {
  Layout l;
  const size_t pairs = (size_t)tokens * top_k;
  l.chunks_d = (int)((d + 127) / 128), l.chunks_f = (int)((f + 127) / 128);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  l.lists = take(sizeof(Lists));
  l.logits = take((size_t)tokens * experts * 4);
  l.x_terms = take((size_t)3 * tokens * l.chunks_d * 256);
  l.a_terms = take((size_t)3 * pairs * l.chunks_f * 256);
  l.products = take(pairs * d * 4);
  l.total = at;
  return l;
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

constexpr int kRouterTokens = 8;  // tokens per CTA of the logits

// CTAs [0, experts * token groups): logits of one expert for up to 8 tokens.  The others: the tokens' terms in
// the order of Pairs, [term][token][unit][register], a thread per unit of 32 columns.
template <typename T, int BITS, int TERMS>
__global__ void __launch_bounds__(256) moe_router_kernel(const T* __restrict__ X, const T* __restrict__ R, int tokens,
                                                         int d, int experts, int router_blocks, int chunks,
                                                         float* __restrict__ logits, uint16_t* __restrict__ terms) {
  if ((int)blockIdx.x < router_blocks) {
    const int e = blockIdx.x % experts, t0 = blockIdx.x / experts * kRouterTokens;
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
    return;
  }
  const int units = d >> 5;
  const int64_t i = (int64_t)(blockIdx.x - router_blocks) * 256 + threadIdx.x;
  if (i >= (int64_t)tokens * units) return;
  const int t = (int)(i / units), u = (int)(i % units);
  float v[32];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float x[8];
    load8<T>(X + (int64_t)t * d + u * 32 + 8 * q, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[8 * q + k] = x[k];
  }
  uint32_t out[TERMS][16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float scale = 1.0f / (float)(1 << Pairs<BITS>::p(r));
    uint16_t lo[TERMS], hi[TERMS];
    split_bf16<TERMS>(v[Pairs<BITS>::lo(r)] * scale, lo);
    split_bf16<TERMS>(v[Pairs<BITS>::hi(r)] * scale, hi);
#pragma unroll
    for (int k = 0; k < TERMS; ++k) out[k][r] = lo[k] | ((uint32_t)hi[k] << 16);
  }
#pragma unroll
  for (int k = 0; k < TERMS; ++k) {
    uint4* dst = reinterpret_cast<uint4*>(terms + ((int64_t)(k * tokens + t) * chunks * 4 + u) * 32);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      dst[q] = make_uint4(out[k][4 * q], out[k][4 * q + 1], out[k][4 * q + 2], out[k][4 * q + 3]);
  }
}

// ------------------------------------------------------------------ top-K and the lists
__device__ __forceinline__ uint32_t ordered(float v) {  // larger float <=> larger integer
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One CTA.  A warp per token chooses its experts (largest logits first, ties to the lowest index) and their
// weights; then every expert's thread collects its pairs in order.
__global__ void __launch_bounds__(1024) moe_route_kernel(const float* __restrict__ logits, int tokens, int experts,
                                                         int top_k, int renormalize, int tile_tokens,
                                                         int32_t* __restrict__ ids, float* __restrict__ weights,
                                                         Lists* __restrict__ lists, int32_t* status) {
  __shared__ int32_t id_of[kMaxPairs];
  __shared__ int32_t first_of[kMaxExperts], tile_of[kMaxExperts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = tokens * top_k;
  if (logits != nullptr) {
    for (int t = warp; t < tokens; t += 32) {
      constexpr int N = kMaxExperts / 32;
      float l[N];
      uint32_t key[N];
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < experts ? logits[(int64_t)t * experts + e] : -INFINITY;
        key[i] = e < experts ? max(ordered(l[i]), 1u) : 0u;  // 0: not there, or chosen before
        mx = fmaxf(mx, l[i]);
      }
      mx = warp_max(mx);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (lane + 32 * i < experts) sum += expf(l[i] - mx);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      float mine = 0.0f, chosen = 0.0f;  // lane k keeps the k-th weight
      for (int k = 0; k < top_k; ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) best = max(best, key[i]);
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (key[i] == top) at = min(at, (uint32_t)(lane + 32 * i));
        const int e = (int)__reduce_min_sync(0xffffffffu, at);
        float le = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (lane + 32 * i == e) le = l[i], key[i] = 0;
        le = __shfl_sync(0xffffffffu, le, e & 31);
        const float w = expf(le - mx) / sum;
        chosen += w;
        if (lane == k) mine = w;
        if (lane == 0) {
          ids[t * top_k + k] = e;
          id_of[t * top_k + k] = e;
        }
      }
      if (lane < top_k) weights[t * top_k + lane] = renormalize ? mine / chosen : mine;
    }
  } else {
    for (int p = threadIdx.x; p < pairs; p += 1024) {
      const int e = ids[p];
      if (e < 0 || e >= experts) report_status(status, GPTQ_ERR_ARG, p);
      id_of[p] = e;
    }
  }
  __syncthreads();
  const int e = threadIdx.x;
  int count = 0;
  if (e < experts) {
    for (int p = 0; p < pairs; ++p) count += id_of[p] == e;
    first_of[e] = count;
    tile_of[e] = (count + tile_tokens - 1) / tile_tokens;
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
  if (e < experts && count > 0) {
    int at = first_of[e];
    for (int p = 0; p < pairs; ++p)
      if (id_of[p] == e) lists->pairs[at++] = p;
    for (int i = 0, left = count; left > 0; ++i, left -= tile_tokens)
      lists->tiles[tile_of[e] + i] = {e, first_of[e] + i * tile_tokens, min(left, tile_tokens)};
  }
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
  int chunks, row_tiles;   // 128-column chunks, work items per tile
  int top_k;
  const uint16_t* terms;   // [term][row][chunk][unit][register]
  int64_t term_stride;
  const Lists* lists;
  uint16_t* out_terms;     // up: terms of the activations [term][pair][...]
  int64_t out_term_stride;
  int out_chunks, out_count;
  float* products;         // down: [pair][rows]
};

// BITS words of a unit
template <int BITS>
__device__ __forceinline__ void load_unit(const uint32_t* p, bool ok, uint32_t (&w)[BITS]) {
#pragma unroll
  for (int i = 0; i < BITS; ++i) w[i] = 0;
  if (!ok) return;
  if constexpr (BITS == 4) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (BITS == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BITS; ++i) w[i] = __ldg(p + i);
  }
}

constexpr int kProductWarps = 8;

// A work item is 32 weight rows (two M tiles of 16: consecutive rows, or the same 16 rows of gate and up) of
// one expert times up to 8 NT of its tokens.  The CTA's warps take the 128-column chunks in turn; in a
// chunk the four lanes of a row take a unit of 32 codes each, all in registers, and the next chunk's words
// are loaded while one is worked on.  After each chunk the sums over 128 columns are scaled into fp32 sums;
// at the end the warps' sums are added in order through shared memory.
// SUB: scales change inside a chunk (groups of 32 or 64); each quarter then has accumulators of its own and
// sees the other quarters' tokens as zeros.
template <int BITS, int TERMS, int NT, int SUB>
__global__ void __launch_bounds__(kProductWarps * 32, 2) moe_product_kernel(const ProductArgs a) {
  __shared__ float sums[kProductWarps][32][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n_items = a.lists->n_tiles * a.row_tiles;
  const int64_t row_words = (int64_t)a.units * BITS;
  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    const Tile tile = a.lists->tiles[item / a.row_tiles];
    const int rt = item % a.row_tiles;
    // this lane's four rows: g and g + 8 of both M tiles
    const uint32_t* words[4];
    const float* scales[4];
    const int32_t* zeros[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool second = i >= 2;
      const Matrix& m = a.mode == kUpGated && second ? a.b : a.a;
      const int row = a.mode == kUpGated ? rt * 16 + g + 8 * (i & 1) : rt * 32 + g + 8 * i;
      const int64_t r = (int64_t)tile.expert * a.rows + row;
      words[i] = m.words + r * row_words;
      scales[i] = m.scales + r * a.ng;
      zeros[i] = m.zeros + r * a.ng;
    }
    // this lane's tokens as a column of B: entry g of every 8
    const uint16_t* tok[NT];
    bool here[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      here[n] = 8 * n + g < tile.count;
      const int p = here[n] ? a.lists->pairs[tile.first + 8 * n + g] : 0;
      tok[n] = a.terms + (int64_t)(a.mode == kDown ? p : p / a.top_k) * a.chunks * 128 + t * 32;
    }
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
    uint32_t next[4][BITS];
    auto load_words = [&](int c) {
      const int u = 4 * c + t;
#pragma unroll
      for (int i = 0; i < 4; ++i) load_unit<BITS>(words[i] + (int64_t)u * BITS, u < a.units, next[i]);
    };
    load_words(warp);
    for (int c = warp; c < a.chunks; c += kProductWarps) {
      const int u = 4 * c + t;
      const bool unit_here = u < a.units;
      const int grid = min(u, a.units - 1) / a.group_units;
      uint32_t v[4][16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unit_pairs<BITS>(next[i], v[i]);
        const int32_t z = __ldg(zeros[i] + grid);
#pragma unroll
        for (int r = 0; r < 16; ++r) v[i][r] = sub_bf16x2(v[i][r], zero_pair<BITS>(z, Pairs<BITS>::p(r)));
      }
      load_words(c + kProductWarps);
      float sum[SUB][2][NT][4];
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[s][m][n][i] = 0.0f;
#pragma unroll
      for (int k = 0; k < TERMS; ++k) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (8 * n >= tile.count) break;
          const uint4* src = reinterpret_cast<const uint4*>(tok[n] + k * a.term_stride + (int64_t)c * 128);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 x = here[n] && unit_here ? __ldg(src + q) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
              for (int s = 0; s < SUB; ++s) {
                const bool mine = SUB == 1 || t == s;
                mma_bf16(sum[s][m][n], v[2 * m][4 * q], v[2 * m + 1][4 * q], v[2 * m][4 * q + 1], v[2 * m + 1][4 * q + 1],
                         mine ? x.x : 0u, mine ? x.y : 0u);
                mma_bf16(sum[s][m][n], v[2 * m][4 * q + 2], v[2 * m + 1][4 * q + 2], v[2 * m][4 * q + 3],
                         v[2 * m + 1][4 * q + 3], mine ? x.z : 0u, mine ? x.w : 0u);
              }
            }
          }
        }
      }
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        const int sg = SUB == 1 ? 4 * c / a.group_units : min(4 * c + s, a.units - 1) / a.group_units;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float s0 = __ldg(scales[2 * m] + sg), s1 = __ldg(scales[2 * m + 1] + sg);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[m][n][0] = fmaf(s0, sum[s][m][n][0], acc[m][n][0]);
            acc[m][n][1] = fmaf(s0, sum[s][m][n][1], acc[m][n][1]);
            acc[m][n][2] = fmaf(s1, sum[s][m][n][2], acc[m][n][2]);
            acc[m][n][3] = fmaf(s1, sum[s][m][n][3], acc[m][n][3]);
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
    auto total = [&](int r, int n) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kProductWarps; ++w) s += sums[w][r][n];
      return s;
    };
    const int out_rows = a.mode == kUpGated ? 16 : 32;
    for (int i = threadIdx.x; i < out_rows * tile.count; i += kProductWarps * 32) {
      const int r = i % out_rows, n = i / out_rows;
      const int p = a.lists->pairs[tile.first + n];
      const int row = rt * out_rows + r;
      if (a.mode == kDown) {
        a.products[(int64_t)p * a.rows + row] = total(r, n);
        continue;
      }
      float h;
      if (a.mode == kUpGated) {
        const float gate = total(r, n);
        h = gate / (1.0f + expf(-gate)) * total(16 + r, n);
      } else {
        h = total(r, n);
        h = h < 0.0f ? 0.0f : h;  // NaN stays
      }
      // its place among the next product's columns
      const int j = row & 31;
      const int reg = Pairs<BITS>::reg(j);
      uint16_t terms[3];
      split_bf16<3>(h * (1.0f / (float)(1 << Pairs<BITS>::p(reg))), terms);
      uint16_t* dst = a.out_terms + ((int64_t)p * a.out_chunks * 4 + (row >> 5)) * 32 + 2 * reg + Pairs<BITS>::half(j);
      for (int k = 0; k < a.out_count; ++k) dst[k * a.out_term_stride] = terms[k];
    }
  }
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
template <int BITS, int TERMS>
gptq_status launch_product(const ProductArgs& a, int nt, bool sub, int max_tiles, int sms, cudaStream_t s) {
  const int64_t items = (int64_t)max_tiles * a.row_tiles;
  const int grid = (int)std::min<int64_t>(items, 2 * (int64_t)sms);
  if (sub)
    moe_product_kernel<BITS, TERMS, 1, 4><<<grid, kProductWarps * 32, 0, s>>>(a);
  else if (nt == 1)
    moe_product_kernel<BITS, TERMS, 1, 1><<<grid, kProductWarps * 32, 0, s>>>(a);
  else
    moe_product_kernel<BITS, TERMS, 4, 1><<<grid, kProductWarps * 32, 0, s>>>(a);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <int BITS>
gptq_status launch_product_terms(int terms, const ProductArgs& a, int nt, bool sub, int max_tiles, int sms,
                                 cudaStream_t s) {
  switch (terms) {
    case 1: return launch_product<BITS, 1>(a, nt, sub, max_tiles, sms, s);
    case 2: return launch_product<BITS, 2>(a, nt, sub, max_tiles, sms, s);
    default: return launch_product<BITS, 3>(a, nt, sub, max_tiles, sms, s);
  }
}

template <typename T, int BITS, int TERMS>
gptq_status launch_router(const void* X, const void* R, int tokens, int d, int experts, int chunks, float* logits,
                          uint16_t* terms, cudaStream_t s) {
  const int router_blocks = R ? experts * ((tokens + kRouterTokens - 1) / kRouterTokens) : 0;
  const int layout_blocks = (int)(((int64_t)tokens * (d / 32) + 255) / 256);
  moe_router_kernel<T, BITS, TERMS><<<router_blocks + layout_blocks, 256, 0, s>>>(
      static_cast<const T*>(X), static_cast<const T*>(R), tokens, d, experts, router_blocks, chunks, logits, terms);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <int BITS>
gptq_status moe_typed(const MoeArgs& m, cudaStream_t s) {
  const Layout l = layout_of(m.tokens, m.d, m.f, m.experts, m.top_k);
  char* ws = static_cast<char*>(m.workspace);
  Lists* lists = reinterpret_cast<Lists*>(ws + l.lists);
  float* logits = reinterpret_cast<float*>(ws + l.logits);
  uint16_t* x_terms = reinterpret_cast<uint16_t*>(ws + l.x_terms);
  uint16_t* a_terms = reinterpret_cast<uint16_t*>(ws + l.a_terms);
  float* products = reinterpret_cast<float*>(ws + l.products);
  int dev = 0, sms = 0;
  GPTQ_CUDA_TRY(cudaGetDevice(&dev));
  GPTQ_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  const int tokens = (int)m.tokens, d = (int)m.d, f = (int)m.f;
  const int pairs = tokens * m.top_k;
  const int x_count = m.x_dtype == GPTQ_BF16 ? 1 : (m.x_dtype == GPTQ_FP16 ? 2 : 3);
  const int a_count = m.y_dtype == GPTQ_FP32 ? 3 : 2;
  gptq_status st;
  switch (m.x_dtype) {
    case GPTQ_BF16: st = launch_router<__nv_bfloat16, BITS, 1>(m.X, m.router, tokens, d, m.experts, l.chunks_d, logits, x_terms, s); break;
    case GPTQ_FP16: st = launch_router<__half, BITS, 2>(m.X, m.router, tokens, d, m.experts, l.chunks_d, logits, x_terms, s); break;
    default: st = launch_router<float, BITS, 3>(m.X, m.router, tokens, d, m.experts, l.chunks_d, logits, x_terms, s); break;
  }
  if (st != GPTQ_OK) return st;
  // up to 8 tokens an expert's list is one N tile; longer lists go 32 at a time so that the codes are taken
  // apart once for four N tiles (scales that change inside a chunk need the registers: 8 at a time)
  const bool sub = m.group_size == 32 || m.group_size == 64;
  const int nt = pairs <= 8 || sub ? 1 : 4;
  const int tile_tokens = 8 * nt;
  const int max_tiles = std::min(pairs, std::min(m.experts, pairs) + pairs / tile_tokens);
  moe_route_kernel<<<1, 1024, 0, s>>>(m.router ? logits : nullptr, tokens, m.experts, m.top_k, m.renormalize,
                                      tile_tokens, m.ids, m.weights, lists, m.status);
  GPTQ_LAUNCH_CHECK();
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
  a.chunks = l.chunks_d, a.row_tiles = m.gated ? f / 16 : f / 32;
  a.top_k = m.top_k;
  a.terms = x_terms, a.term_stride = (int64_t)tokens * l.chunks_d * 128;
  a.lists = lists;
  a.out_terms = a_terms, a.out_term_stride = (int64_t)pairs * l.chunks_f * 128;
  a.out_chunks = l.chunks_f, a.out_count = a_count;
  st = launch_product_terms<BITS>(x_count, a, nt, sub, max_tiles, sms, s);
  if (st != GPTQ_OK) return st;
  a.mode = kDown;
  a.a = matrix(m.down);
  a.rows = d, a.units = f / 32;
  a.ng = m.group_size ? f / m.group_size : 1;
  a.group_units = m.group_size ? m.group_size / 32 : a.units;
  a.chunks = l.chunks_f, a.row_tiles = d / 32;
  a.terms = a_terms, a.term_stride = (int64_t)pairs * l.chunks_f * 128;
  a.products = products;
  st = launch_product_terms<BITS>(a_count, a, nt, sub, max_tiles, sms, s);
  if (st != GPTQ_OK) return st;
  const unsigned blocks = (unsigned)(((int64_t)tokens * d + 255) / 256);
  switch (m.y_dtype) {
    case GPTQ_BF16: moe_combine_kernel<<<blocks, 256, 0, s>>>(products, m.ids, m.weights, tokens, d, m.top_k, m.experts, static_cast<__nv_bfloat16*>(m.Y)); break;
    case GPTQ_FP16: moe_combine_kernel<<<blocks, 256, 0, s>>>(products, m.ids, m.weights, tokens, d, m.top_k, m.experts, static_cast<__half*>(m.Y)); break;
    default: moe_combine_kernel<<<blocks, 256, 0, s>>>(products, m.ids, m.weights, tokens, d, m.top_k, m.experts, static_cast<float*>(m.Y)); break;
  }
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace

size_t moe_workspace(int64_t tokens, int64_t d, int64_t f, int64_t experts, int64_t top_k) {
  return layout_of(tokens, d, f, experts, top_k).total;
}

gptq_status moe_launch(const MoeArgs& m, int32_t bits, cudaStream_t stream) {
  switch (bits) {
    case 2: return moe_typed<2>(m, stream);
    case 3: return moe_typed<3>(m, stream);
    default: return moe_typed<4>(m, stream);
  }
}

}  // namespace gptq
