// Y = A B^T for e4m3 operands with an fp32 scale per row (or 128 rows) and block of 128 columns:
//   Y[i, j] = sum_b a_scales[i, b] b_scales[j / rows, b] P_b[i, j],   P_b[i, j] = sum_{t in block b} A[i, t] B[j, t].
//
// The scales change every 128 columns, so the tensor cores can only carry the sum inside one block: each
// P_b is a fresh accumulator in TMEM, and the scaled sum over b runs in fp32 registers of the epilogue
// warps while the MMAs of the next blocks proceed into the other accumulators.  Weights (B) take the
// M side of the MMA, tokens (A) the N side: a TMEM lane is a weight row, so its scale is one register per
// thread and block, the tokens' scales come from shared memory as a vector common to all lanes
// (two fp32x2 operations per two products), and a handful of tokens costs a tile 16 columns wide, not 128.
//
// One CTA per SM, persistent.  A unit is a tile of 128 weight rows x NT tokens and a range of blocks:
//   warp 0      TMA producer: ring of stages, one block (128 bytes of every row) each
//   warp 1      tcgen05.mma kind::f8f6f4 issuer (one thread) and TMEM owner: four K = 32 steps per block
//   warps 2-9   epilogue: 32 rows x NT / 2 tokens per warp
// Every mbarrier wait is bounded; on a timeout the kernel records GPTQ_ERR_TIMEOUT, the other roles
// leave, copies and MMAs in flight land, TMEM is freed.
#include <algorithm>

#include "kernels.h"
#include "tc_common.cuh"

namespace gptq {
namespace {

using namespace tc;

constexpr int BM = 128;           // weight rows per tile
constexpr int BK = 128;           // columns per block (and per stage): 128 bytes, one swizzle row
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + EPI_WARPS * 32;
constexpr int SG = 8;             // blocks whose token scales are staged at a time
constexpr int kPlanSMs = 148;
constexpr int kGroupTiles = 16;   // weight tiles walked together (see unit_coords)
constexpr int kSmemBudget = 200 * 1024;

template <int NT>
struct Cfg {
  static constexpr int kStageBytes = (BM + NT) * BK;
  static constexpr int kStages = kSmemBudget / kStageBytes > 10 ? 10 : kSmemBudget / kStageBytes;
  static constexpr int kAccs = NT >= 256 ? 2 : 4;  // accumulators in TMEM
  static constexpr int kTmemCols = NT * kAccs < 32 ? 32 : NT * kAccs;
  static constexpr int kCols = NT / 2;  // tokens per epilogue thread
  static constexpr int kScaleBytes = 2 * SG * NT * 4;
  static constexpr int kSmem = kStages * kStageBytes + kScaleBytes + 1024 + 512;
};

struct Args {
  int m, n, kb;                    // tokens, weight rows, blocks
  int tiles_w, tiles_t, units;     // weight tiles, token tiles, work units
  int kb_per_split;
  int b_shift;                     // weight row -> row of b_scales: 0 or 7
  uint32_t idesc;
  const float* a_scales;
  const float* b_scales;
  void* Y;
  float* partial;                  // [split][m][n] when the blocks are split, else null
  int32_t* status;
};

__device__ __forceinline__ void umma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 8 or 16 consecutive TMEM columns of this warp's 32 lanes; the values are there after tmem_wait()
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]);
template <>
__device__ __forceinline__ void tmem_ld<8>(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  lo = __uint_as_float(a), hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// unit -> (weight tile, token tile, split).  Weight tiles are walked in groups of kGroupTiles, all token
// tiles for each group, so that the tiles in flight share few rows of either operand in L2.
__device__ __forceinline__ void unit_coords(int u, const Args& a, int& tw, int& tt, int& s) {
  const int tiles = a.tiles_w * a.tiles_t;
  s = u / tiles;
  const int t = u % tiles;
  const int g = t / (kGroupTiles * a.tiles_t);
  const int w = min(kGroupTiles, a.tiles_w - g * kGroupTiles);
  const int r = t - g * kGroupTiles * a.tiles_t;
  tw = g * kGroupTiles + r % w;
  tt = r / w;
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <int NT, typename TY>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_t,
                      const Args a) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* token_scales = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);  // [2][SG][NT]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes + C::kScaleBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + C::kAccs;
  uint64_t* drain = acc_empty + C::kAccs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kAccs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      uint32_t stage = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
        int tw, tt, s;
        unit_coords(u, a, tw, tt, s);
        const int b0 = s * a.kb_per_split, b1 = min(a.kb, b0 + a.kb_per_split);
        for (int b = b0; b < b1; ++b, ++stage) {
          const uint32_t slot = stage % C::kStages, round = stage / C::kStages;
          if (!mbar_wait(&empty[slot], (round & 1) ^ 1, abort_flag, a.status, 51)) {
            ok = false;
            break;
          }
          uint8_t* W = smem + slot * C::kStageBytes;
          mbar_expect_tx(&full[slot], C::kStageBytes);
          tma_load_2d(W, &map_w, b * BK, tw * BM, &full[slot]);
          tma_load_2d(W + BM * BK, &map_t, b * BK, tt * NT, &full[slot]);
        }
      }
      if (!ok) {  // let the copies already issued land before the CTA leaves
        const uint32_t first = stage > C::kStages ? stage - C::kStages : 0;
        for (uint32_t i = first; i < stage; ++i) mbar_wait_drain(&full[i % C::kStages], (i / C::kStages) & 1);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      uint32_t stage = 0;  // blocks issued so far: stage slot and accumulator follow from it
      bool ok = true;
      const uint32_t smem0 = smem_u32(smem);
      for (int u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
        int tw, tt, s;
        unit_coords(u, a, tw, tt, s);
        const int nb = min(a.kb, (s + 1) * a.kb_per_split) - s * a.kb_per_split;
        for (int b = 0; b < nb; ++b, ++stage) {
          const uint32_t buf = stage % C::kAccs, use = stage / C::kAccs;
          const uint32_t slot = stage % C::kStages, round = stage / C::kStages;
          if (!mbar_wait(&acc_empty[buf], (use & 1) ^ 1, abort_flag, a.status, 52) ||
              !mbar_wait(&full[slot], round & 1, abort_flag, a.status, 53)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // K-major rows of 128 bytes with the 128-byte swizzle; a step of 32 columns is 32 bytes
          const uint64_t wd = sdesc_sw128(smem0 + slot * C::kStageBytes, 16, 1024);
          const uint64_t td = sdesc_sw128(smem0 + slot * C::kStageBytes + BM * BK, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            umma_f8(tmem_base + buf * NT, wd + (uint64_t)(kk * 2), td + (uint64_t)(kk * 2), a.idesc, kk > 0 ? 1u : 0u);
          umma_commit(&empty[slot]);
          umma_commit(&acc_full[buf]);
        }
      }
      // all MMAs issued by this thread are complete before TMEM is released
      umma_commit(drain);
      mbar_wait_drain(drain, 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue
    const int ew = warp - 2;
    const int quad = warp & 3;  // TMEM lanes this warp may access: 32*quad .. 32*quad+31
    const int half = ew >> 2;   // tokens NT/2*half .. of the tile
    const int et = threadIdx.x - 64;
    constexpr int LD = C::kCols < 16 ? 8 : 16;  // TMEM columns per load
    constexpr int TPT = (NT + EPI_WARPS * 32 - 1) / (EPI_WARPS * 32);  // tokens whose scales a thread stages
    static_assert(TPT == 1, "one token per epilogue thread");
    uint32_t stage = 0, group = 0;
    // After a wait that gave up the warp stops waiting and storing but still walks its units, because all
    // eight warps have to meet at the named barrier.
    bool ok = true;
    for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
      int tw, tt, s;
      unit_coords(u, a, tw, tt, s);
      const int b0 = s * a.kb_per_split, b1 = min(a.kb, b0 + a.kb_per_split);
      const int row = tw * BM + 32 * quad + lane;  // this thread's weight row
      const int t0 = tt * NT;
      const float* wsc = a.b_scales + (int64_t)(min(row, a.n - 1) >> a.b_shift) * a.kb;
      const bool stages_scales = et < NT;
      const float* tsc = a.a_scales + (int64_t)min(t0 + min(et, NT - 1), a.m - 1) * a.kb;
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int c = 0; c < C::kCols / 2; ++c) acc[c] = 0ull;
      float w_next = __ldg(wsc + b0);
      for (int g0 = b0; g0 < b1; g0 += SG, ++group) {
        // the scales of this tile's tokens for SG blocks, [block][token]; the other buffer may still be read
        float* sc = token_scales + (group & 1) * SG * NT;
        if (stages_scales) {
#pragma unroll
          for (int i = 0; i < SG; ++i) sc[i * NT + et] = g0 + i < b1 ? __ldg(tsc + g0 + i) : 0.0f;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(EPI_WARPS * 32) : "memory");
        const int g1 = min(b1, g0 + SG);
        for (int b = g0; b < g1; ++b, ++stage) {
          const uint32_t buf = stage % C::kAccs, use = stage / C::kAccs;
          const float w = w_next;
          if (b + 1 < b1) w_next = __ldg(wsc + b + 1);
          const uint64_t w2 = pack2(__float_as_uint(w), __float_as_uint(w));
          const float* scb = sc + (b - g0) * NT + half * C::kCols;
          if (ok) ok = mbar_wait(&acc_full[buf], use & 1, abort_flag, a.status, 54);
          tc_fence_after();
          const uint32_t taddr = tmem_base + ((uint32_t)(32 * quad) << 16) + buf * NT + half * C::kCols;
#pragma unroll
          for (int q = 0; q < C::kCols / LD; ++q) {
            uint32_t v[LD];
            tmem_ld<LD>(taddr + LD * q, v);
            tmem_wait();
#pragma unroll
            for (int i = 0; i < LD; i += 4) {
              const ulonglong2 ts = *reinterpret_cast<const ulonglong2*>(scb + LD * q + i);
              const int c = (LD * q + i) / 2;
              acc[c] = fma2(mul2(pack2(v[i], v[i + 1]), ts.x), w2, acc[c]);
              acc[c + 1] = fma2(mul2(pack2(v[i + 2], v[i + 3]), ts.y), w2, acc[c + 1]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
      }
      if (ok && row < a.n) {
        const int tok0 = t0 + half * C::kCols;
#pragma unroll
        for (int c = 0; c < C::kCols; c += 2) {
          float v0, v1;
          unpack2(acc[c / 2], v0, v1);
          if (a.partial == nullptr) {
            TY* y = static_cast<TY*>(a.Y) + (int64_t)(tok0 + c) * a.n + row;
            if (tok0 + c < a.m) y[0] = from_f32<TY>(v0);
            if (tok0 + c + 1 < a.m) y[a.n] = from_f32<TY>(v1);
          } else {
            float* y = a.partial + ((int64_t)s * a.m + tok0 + c) * a.n + row;
            if (tok0 + c < a.m) y[0] = v0;
            if (tok0 + c + 1 < a.m) y[a.n] = v1;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// Y = the splits' partial sums, added in split order.
template <typename TY>
__global__ void __launch_bounds__(256) fp8_matmul_reduce_kernel(const float* __restrict__ partial, int splits,
                                                                int64_t n, TY* __restrict__ Y) {
  for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
    float s = 0.0f;
    for (int t = 0; t < splits; ++t) s += partial[t * n + e];
    Y[e] = from_f32<TY>(s);
  }
}

struct Plan {
  int nt, tiles_w, tiles_t, kb, kb_per_split, splits;
};

// Tile width and split of the blocks with the lowest estimated time in cycles: a block costs an SM about
// 330 + 2.6 NT (its operands' way through shared memory), a unit 1500 for its fill and its epilogue, and
// split sums are written and read back at about 3000 bytes per cycle of the whole GPU plus a launch.
Plan make_plan(int64_t m, int64_t n, int64_t k) {
  Plan best = {};
  double best_cost = 1e300;
  const int kb = (int)((k + BK - 1) / BK);
  for (int nt = 16; nt <= 256; nt *= 2) {
    const int64_t tw = (n + BM - 1) / BM, tt = (m + nt - 1) / nt;
    for (int want = 1; want <= 16 && want <= kb; ++want) {
      const int per = (kb + want - 1) / want, splits = (kb + per - 1) / per;
      if (splits != want) continue;
      const int64_t units = tw * tt * splits;
      if (splits > 1 && units > 2 * kPlanSMs) continue;
      const double waves = (double)((units + kPlanSMs - 1) / kPlanSMs);
      double cost = waves * (per * (330.0 + 2.6 * nt) + 1500.0);
      if (splits > 1) cost += 8.0 * splits * (double)m * (double)n / 3000.0 + 4000.0;
      if (cost < best_cost) {
        best_cost = cost;
        best = {nt, (int)tw, (int)tt, kb, per, splits};
      }
    }
  }
  return best;
}

// [rows, k] bytes in boxes of box_rows x 128 with the 128-byte swizzle; rows and columns past the edges read 0
bool operand_map(CUtensorMap* map, const void* base, int64_t rows, int64_t k, int box_rows) {
  auto encode = encode_fn();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)k};
  const cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)box_rows};
  const cuuint32_t elem[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, elem,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, typename TY>
gptq_status launch(const CUtensorMap& w, const CUtensorMap& t, Args a, int sms, cudaStream_t s) {
  // D fp32 (bit 4), A and B e4m3 (0), both K-major, N = NT, M = 128
  a.idesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
  GPTQ_CUDA_TRY(cudaFuncSetAttribute(fp8_matmul_kernel<NT, TY>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Cfg<NT>::kSmem));
  fp8_matmul_kernel<NT, TY><<<std::min(a.units, sms), THREADS, Cfg<NT>::kSmem, s>>>(w, t, a);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <typename TY>
gptq_status launch_typed(const Plan& p, const CUtensorMap& w, const CUtensorMap& t, const Args& a, int sms,
                         cudaStream_t s) {
  gptq_status st;
  switch (p.nt) {
    case 16: st = launch<16, TY>(w, t, a, sms, s); break;
    case 32: st = launch<32, TY>(w, t, a, sms, s); break;
    case 64: st = launch<64, TY>(w, t, a, sms, s); break;
    case 128: st = launch<128, TY>(w, t, a, sms, s); break;
    default: st = launch<256, TY>(w, t, a, sms, s); break;
  }
  if (st != GPTQ_OK || a.partial == nullptr) return st;
  const int64_t e = (int64_t)a.m * a.n;
  const unsigned blocks = (unsigned)std::min<int64_t>((e + 255) / 256, kPlanSMs * 8);
  fp8_matmul_reduce_kernel<TY><<<blocks, 256, 0, s>>>(a.partial, p.splits, e, static_cast<TY*>(a.Y));
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace

size_t fp8_matmul_workspace(int64_t m, int64_t n, int64_t k) {
  const Plan p = make_plan(m, n, k);
  return p.splits > 1 ? align_up((size_t)p.splits * m * n * sizeof(float), 256) : 0;
}

gptq_status fp8_matmul_launch(const void* A, const float* a_scales, const void* B, const float* b_scales,
                              int32_t b_block_rows, int64_t m, int64_t n, int64_t k, void* Y, int32_t y_dtype,
                              int32_t* status, void* workspace, cudaStream_t stream) {
  const Plan p = make_plan(m, n, k);
  const int64_t units = (int64_t)p.tiles_w * p.tiles_t * p.splits;
  if (units > 0x7fffffff - kPlanSMs) return GPTQ_ERR_ARG;
  CUtensorMap w, t;
  if (!operand_map(&w, B, n, k, BM) || !operand_map(&t, A, m, k, p.nt)) return GPTQ_ERR_CUDA;
  int dev = 0, sms = 0;
  GPTQ_CUDA_TRY(cudaGetDevice(&dev));
  GPTQ_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  Args a = {};
  a.m = (int)m, a.n = (int)n, a.kb = p.kb;
  a.tiles_w = p.tiles_w, a.tiles_t = p.tiles_t, a.units = (int)units;
  a.kb_per_split = p.kb_per_split;
  a.b_shift = b_block_rows == 128 ? 7 : 0;
  a.a_scales = a_scales, a.b_scales = b_scales;
  a.Y = Y;
  a.partial = p.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  a.status = status;
  switch (y_dtype) {
    case GPTQ_BF16: return launch_typed<__nv_bfloat16>(p, w, t, a, sms, stream);
    case GPTQ_FP16: return launch_typed<__half>(p, w, t, a, sms, stream);
    default: return launch_typed<float>(p, w, t, a, sms, stream);
  }
}

}  // namespace gptq
