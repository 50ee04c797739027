// Y = A B^T for e4m3 operands with an fp32 scale per row (or 128 rows) and block of 128 columns:
//   Y[i, j] = sum_b a_scales[i, b] b_scales[j / rows, b] P_b[i, j],   P_b[i, j] = sum_{t in block b} A[i, t] B[j, t].
//
// The scales change every 128 columns, so the tensor cores can only carry the sum inside one block: each
// P_b is a fresh accumulator in TMEM, and the scaled sum over b runs in fp32 registers of the epilogue
// warps while the MMAs of the next blocks proceed into the other accumulators.  The epilogue reads TMEM
// in the 16x256b shape: a thread holds four token rows and column pairs, so a block costs it four row
// scales and, where every weight row has its own scale, one 8-byte shared-memory load per 8 columns of
// the warp.  (In the 32x32b shape, a row per thread, the column scales are the same for all lanes, and
// those broadcast loads alone took over 1000 shared-memory cycles per 128 x 256 block: 8192 x 11008 x 4096
// with a scale per weight row took 683 us instead of 480.)  Two fp32x2 operations per two products, or one where 128 weight rows share a scale,
// which is then multiplied into the row scales.
//
// One CTA per SM, persistent.  A unit is a tile of 128 tokens x NT weight rows and a range of blocks:
//   warp 0      TMA producer: ring of stages, one block (128 bytes of every row) each
//   warp 1      tcgen05.mma kind::f8f6f4 issuer (one thread) and TMEM owner: four K = 32 steps per block
//   warps 4-11  epilogue: 32 tokens x NT / 2 weight rows per warp
// Every mbarrier wait is bounded; on a timeout the kernel records GPTQ_ERR_TIMEOUT, the other roles
// leave, copies and MMAs in flight land, TMEM is freed.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "tc_common.cuh"

namespace gptq {
namespace {

using namespace tc;

constexpr int BM = 128;           // tokens per tile
constexpr int BK = 128;           // columns per block (and per stage): 128 bytes, one swizzle row
constexpr int SG = 4;             // blocks whose token scales are staged at a time
constexpr int kPlanSMs = 148;
constexpr int kGroupTiles = 16;   // token tiles walked together (see unit_coords)
constexpr int kSmemBudget = 200 * 1024;

template <int NT>
struct Cfg {
  static constexpr int kEpiWarps = 8;
  static constexpr int kEpiThreads = kEpiWarps * 32;
  static constexpr int kThreads = 128 + kEpiThreads;
  static constexpr int kStageBytes = (BM + NT) * BK;
  static constexpr int kStages = kSmemBudget / kStageBytes > 10 ? 10 : kSmemBudget / kStageBytes;
  static constexpr int kAccs = 4;  // accumulators in TMEM
  static constexpr int kAccCols = NT == 96 ? 128 : NT;  // from one to the next: TMEM comes in powers of two
  static constexpr int kTmemCols = kAccCols * kAccs;
  static constexpr int kCols = NT * 4 / kEpiWarps;  // weight rows per epilogue warp
  static constexpr int kScaleRow = BM + NT;  // staged scales per block
  static constexpr int kScaleBytes = 2 * SG * kScaleRow * 4;
  static constexpr int kSmem = kStages * kStageBytes + kScaleBytes + 1024 + 512;
};

struct Args {
  int m, n, kb;                    // tokens, weight rows, blocks
  int tiles_t, tiles_w, units;     // token tiles, weight tiles, work units
  int kb_per_split;
  int scale_width;                 // floats per load that the scales' rows are aligned for: 1, 2 or 4
  bool vec_y, pair_y;              // Y's rows start on 16 bytes, on pairs of values
  int token_bytes;                 // bytes of a stage's token box (fewer than 128 rows when m is small)
  uint32_t idesc;
  const float* a_scales;
  const float* b_scales;
  void* Y;
  float* partial;                  // [split][m][ld] when the blocks are split, else null
  int ld, splits;
  int32_t* status;
};

// One lane of a converged warp.  The producer's and the issuers' loops run in whole warps with only the TMA, MMA and
// commit instructions under this predicate: their operands then stay in the warp's uniform registers.  With the
// loops inside `if (lane == 0)` every operand was moved there first, and a block's four MMAs and two commits
// took their thread 730 cycles, more than the tensor core needs for them.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// position in a ring of N slots: the slot, and the parity of the round
template <int N>
struct Ring {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, parity ^= 1;
  }
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

// 16 TMEM lanes x 8 J columns: r[4 j + {0, 1}] are columns 8 j + 2 (lane % 4) + {0, 1} of row lane / 4,
// r[4 j + {2, 3}] the same columns of row lane / 4 + 8; there after tmem_wait()
template <int J>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r);
template <>
__device__ __forceinline__ void tmem_ld<4>(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
template <>
__device__ __forceinline__ void tmem_ld<2>(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
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

// unit -> (token tile, weight tile, split).  Token tiles are walked in groups of kGroupTiles, all weight
// tiles for each group, so that the tiles in flight share few rows of either operand in L2.
__device__ __forceinline__ void unit_coords(int u, const Args& a, int& tt, int& tw, int& s) {
  const int tiles = a.tiles_w * a.tiles_t;
  s = u / tiles;
  const int t = u % tiles;
  const int g = t / (kGroupTiles * a.tiles_w);
  const int w = min(kGroupTiles, a.tiles_t - g * kGroupTiles);
  const int r = t - g * kGroupTiles * a.tiles_w;
  tt = g * kGroupTiles + r % w;
  tw = r / w;
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// two neighbouring results of a row; `pair`: both exist and y is aligned for both
template <typename T>
__device__ __forceinline__ void store_pair(T* y, float v0, float v1, int left, bool pair) {
  if (pair) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float2*>(y) = make_float2(v0, v1);
    } else {
      T h[2] = {from_f32<T>(v0), from_f32<T>(v1)};
      *reinterpret_cast<uint32_t*>(y) = *reinterpret_cast<uint32_t*>(h);
    }
  } else {
    if (left > 0) y[0] = from_f32<T>(v0);
    if (left > 1) y[1] = from_f32<T>(v1);
  }
}

// NC consecutive results of one row, `left` of which exist
template <int NC, typename T>
__device__ __forceinline__ void store_row(const uint64_t (&acc)[NC / 2], T* y, int left) {
#pragma unroll
  for (int c = 0; c < NC; c += 2) {
    float v0, v1;
    unpack2(acc[c / 2], v0, v1);
    if (c < left) y[c] = from_f32<T>(v0);
    if (c + 1 < left) y[c + 1] = from_f32<T>(v1);
  }
}

// Scales of blocks g0 .. g0 + 3 of one row of kb (past its end: some of its others, which nobody uses), V at a time:
// rows start on 4 V bytes, g0 is a multiple of 4.  One row's scales are kb floats away from the next row's, so every
// lane reads a line of its own: one 16-byte load takes a quarter of four 4-byte loads' time in the load unit.
// The loads are volatile and without conditions so that they stay where they are written, a group of blocks before
// their use, and go straight into the registers that are used: moved down by the compiler, or merged with
// zeros behind a condition, they cost their latency, some 700 cycles a group.
template <int V>
__device__ __forceinline__ void fetch_scales(const float* row, int g0, int kb, float (&v)[4]) {
  if constexpr (V == 4) {
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "l"(row + min(g0, kb - 4)));
  } else if constexpr (V == 2) {
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      asm volatile("ld.global.nc.v2.f32 {%0, %1}, [%2];" : "=f"(v[i]), "=f"(v[i + 1]) : "l"(row + min(g0 + i, kb - 2)));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v[i]) : "l"(row + min(g0 + i, kb - 1)));
  }
}

template <int NT, bool BLOCK, int VEC, typename TY>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_t, const __grid_constant__ CUtensorMap map_w,
                      const Args a) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* token_scales = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);  // [2][SG][kScaleRow]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes + C::kScaleBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + C::kAccs;
  uint64_t* drain = acc_empty + C::kAccs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x / 32), 0), lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kAccs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::kEpiWarps);
    }
    mbar_init(drain, 2);
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
    Ring<C::kStages> r;
    uint32_t issued = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
      int tt, tw, s;
      unit_coords(u, a, tt, tw, s);
      const int b0 = s * a.kb_per_split, b1 = min(a.kb, b0 + a.kb_per_split);
      for (int b = b0; b < b1; ++b, ++issued, r.next()) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[r.slot], r.parity ^ 1, abort_flag, a.status, 51));
        if (!ok) break;
        if (elect_one()) {
          uint8_t* T = smem + r.slot * C::kStageBytes;
          mbar_expect_tx(&full[r.slot], (uint32_t)a.token_bytes + NT * BK);
          tma_load_2d(T, &map_t, b * BK, tt * BM, &full[r.slot]);
          tma_load_2d(T + BM * BK, &map_w, b * BK, tw * NT, &full[r.slot]);
        }
        __syncwarp();
      }
    }
    if (!ok) {  // let the copies already issued land before the CTA leaves
      const uint32_t first = issued > C::kStages ? issued - C::kStages : 0;
      for (uint32_t i = first; i < issued; ++i) mbar_wait_drain(&full[i % C::kStages], (i / C::kStages) & 1);
    }
  } else if (warp < 3) {
    // ---------------------------------------------------------------- MMA issuers: even and odd blocks
    Ring<C::kStages> r;
    Ring<C::kAccs> acc;
    uint32_t mine = warp - 1;  // 0: this block is this warp's
    bool ok = true;
    const uint64_t desc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
    for (int u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
      int tt, tw, s;
      unit_coords(u, a, tt, tw, s);
      const int nb = min(a.kb, (s + 1) * a.kb_per_split) - s * a.kb_per_split;
      for (int b = 0; b < nb; ++b, r.next(), acc.next(), mine ^= 1) {
        if (mine) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty[acc.slot], acc.parity ^ 1, abort_flag, a.status, 52) &&
                                         mbar_wait(&full[r.slot], r.parity, abort_flag, a.status, 53));
        if (!ok) break;
        tc_fence_after();
        // K-major rows of 128 bytes with the 128-byte swizzle; a step of 32 columns is 32 bytes.  Token rows
        // that the box does not reach hold what was there before: they only reach accumulator rows
        // that nobody reads.
        if (elect_one()) {
          const uint64_t td = desc0 + (uint64_t)((r.slot * C::kStageBytes) >> 4);
          const uint64_t wd = td + (uint64_t)((BM * BK) >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            umma_f8(tmem_base + acc.slot * C::kAccCols, td + (uint64_t)(kk * 2), wd + (uint64_t)(kk * 2), a.idesc, kk > 0 ? 1u : 0u);
          umma_commit(&acc_full[acc.slot]);
          umma_commit(&empty[r.slot]);
        }
        __syncwarp();
      }
    }
    // all MMAs issued by this warp are complete before TMEM is released
    if (elect_one()) umma_commit(drain);
    __syncwarp();
    mbar_wait_drain(drain, 0);
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int quad = warp & 3;         // TMEM lanes this warp may access: 32*quad .. 32*quad+31
    const int part = (warp - 4) >> 2;  // columns kCols * part .. of the tile
    const int et = threadIdx.x - 128;
    const int r4 = lane >> 2, c4 = 2 * (lane & 3);  // this thread's rows r4 + 8 i and columns c4 + 8 j + {0, 1}
    constexpr int NQ = (C::kCols + 31) / 32;  // loads per block: 32 columns each, the last one what is left (16 or 32)
    constexpr int SR = C::kScaleRow;
    uint32_t group = 0;
    Ring<C::kAccs> at;  // the accumulator of the block in hand
    // After a wait that gave up the warp stops waiting and storing but still walks its units, because all
    // eight warps have to meet at the named barrier.
    bool ok = true;
    for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
      int tt, tw, s;
      unit_coords(u, a, tt, tw, s);
      const int b0 = s * a.kb_per_split, b1 = min(a.kb, b0 + a.kb_per_split);
      const int t0 = tt * BM, w0 = tw * NT;
      // Scales are staged SG blocks at a time: the first half of the threads the tokens', the second half the weight
      // rows'.  BLOCK: the first half both, multiplied (the tile's weight rows lie in one block of 128).
      const int row = et & 127;
      const float* tsc = a.a_scales + (int64_t)min(t0 + row, a.m - 1) * a.kb;
      const float* wsc = BLOCK ? a.b_scales + (int64_t)(w0 >> 7) * a.kb
                               : a.b_scales + (int64_t)min(w0 + min(row, NT - 1), a.n - 1) * a.kb;
      float t_next[SG], w_next[SG];  // the scales of the group to come
      auto fetch = [&](int g0) {
        if (part == 0) fetch_scales<VEC>(tsc, g0, a.kb, t_next);
        if (BLOCK ? part == 0 : part == 1) fetch_scales<VEC>(wsc, g0, a.kb, w_next);
      };
      fetch(b0);
      const bool rows_here = t0 + 32 * quad < a.m;  // else the warp only keeps the barriers going
      uint64_t acc[4][C::kCols / 8];  // [row r4 + 8 i][column group j]
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < C::kCols / 8; ++j) acc[i][j] = 0ull;
      for (int g0 = b0; g0 < b1; g0 += SG, ++group) {
        float* sc = token_scales + (group & 1) * SG * SR;  // the other buffer may still be read
#pragma unroll
        for (int i = 0; i < SG; ++i) {
          if (part == 0) sc[i * SR + row] = BLOCK ? t_next[i] * w_next[i] : t_next[i];  // [token], then [weight row]
          if (!BLOCK && part == 1 && row < NT) sc[i * SR + BM + row] = w_next[i];
        }
        fetch(g0 + SG);
        asm volatile("bar.sync 1, %0;" ::"n"(C::kEpiThreads) : "memory");
        const int g1 = min(b1, g0 + SG);
        const float* rsc = sc + 32 * quad + r4;
        const float* csc = sc + BM + part * C::kCols + c4;
        for (int b = g0; b < g1; ++b, rsc += SR, csc += SR) {
          uint64_t rs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t r = __float_as_uint(rsc[8 * i]);
            rs[i] = pack2(r, r);
          }
          if (ok) ok = mbar_wait(&acc_full[at.slot], at.parity, abort_flag, a.status, 54);
          tc_fence_after();
          // Two loads a block, waited for one by one: running them ahead of the sums, across blocks, took longer (a
          // block of 128 x 128 1000 cycles instead of 700).
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const int groups = C::kCols - 32 * q >= 32 ? 4 : 2;  // of 8 columns
            uint32_t v[2][16];  // [16-row half]
            if (rows_here) {
              const uint32_t taddr = tmem_base + ((uint32_t)(32 * quad) << 16) + at.slot * C::kAccCols + part * C::kCols + 32 * q;
              if (groups == 4) {
                tmem_ld<4>(taddr, v[0]);
                tmem_ld<4>(taddr + (16u << 16), v[1]);
              } else {
                tmem_ld<2>(taddr, v[0]);
                tmem_ld<2>(taddr + (16u << 16), v[1]);
              }
              tmem_wait();
            }
            if (q == NQ - 1) {  // the last columns are in registers: the accumulator goes back to the MMAs
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&acc_empty[at.slot]);
              at.next();
            }
            if (!rows_here) continue;
#pragma unroll
            for (int j = 0; j < groups; ++j) {
              uint64_t cs = 0;
              if constexpr (!BLOCK) cs = *reinterpret_cast<const uint64_t*>(csc + 8 * (4 * q + j));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t* p = &v[i >> 1][4 * j + 2 * (i & 1)];
                const uint64_t pp = pack2(p[0], p[1]);
                acc[i][4 * q + j] = fma2(BLOCK ? pp : mul2(pp, cs), rs[i], acc[i][4 * q + j]);
              }
            }
          }
        }
      }
      if (ok && rows_here) {
        const bool even = a.partial || a.pair_y;  // rows start on pairs
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = t0 + 32 * quad + r4 + 8 * i;
          if (tok >= a.m) continue;
          const int w = w0 + part * C::kCols + c4;
          const int64_t at = a.partial ? ((int64_t)s * a.m + tok) * a.ld + w : (int64_t)tok * a.n + w;
#pragma unroll
          for (int j = 0; j < C::kCols / 8; ++j) {
            float v0, v1;
            unpack2(acc[i][j], v0, v1);
            const int left = a.n - w - 8 * j;
            if (a.partial == nullptr)
              store_pair(static_cast<TY*>(a.Y) + at + 8 * j, v0, v1, left, even && left > 1);
            else
              store_pair(a.partial + at + 8 * j, v0, v1, left, even && left > 1);
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

// ------------------------------------------------------------------------------------------------
// CTA-pair form, for products with enough 256 x 256 tiles to fill the GPU.  A cluster of two CTAs computes
// a tile of 256 tokens x 256 weight rows with tcgen05.mma.cta_group::2: each CTA loads its 128 tokens and
// half of the weight rows (32 KB per block, where the single-CTA tile of the same area per SM takes 48 KB
// in and out of shared memory and out of L2).  The tile's columns are two accumulators of 128, each with
// its own barriers and its own four epilogue warps, double-buffered: while one half's warps read their
// sums the MMAs of the other half run, and the two warps of a scheduler wait at different times.
//   BLOCK: a thread holds one token row (32x32b loads), one scale per thread and block
//   else:  four token rows and column pairs (16x256b loads), the weights' scales from shared memory
constexpr int PN = 256;                           // weight rows of a pair's tile
constexpr int P_STAGES = 5;
constexpr int P_STAGE_BYTES = (BM + PN / 2) * BK;  // per CTA
constexpr int P_EPI_WARPS = 8;
constexpr int P_THREADS = 128 + P_EPI_WARPS * 32;
constexpr int P_SG = SG;
constexpr int P_SCALE_ROW = 2 * BM;                // floats per block and half: tokens, then its weight rows
constexpr int P_SCALE_BYTES = 2 * 2 * P_SG * P_SCALE_ROW * 4;  // [half][buffer][block]
constexpr int P_OUT_BYTES = P_EPI_WARPS * 4096;    // a 32-row x 128-byte tile per warp on its way to Y
constexpr int P_SMEM = P_STAGES * P_STAGE_BYTES + P_OUT_BYTES + P_SCALE_BYTES + 1024 + 512;
// register split (per thread): warps 0-3 give theirs up to the epilogue, whose sums take 128
constexpr int kLaunchRegs = 168, kEpiRegs = 232, kOtherRegs = 40;
static_assert(128 * kOtherRegs + P_EPI_WARPS * 32 * kEpiRegs <= P_THREADS * kLaunchRegs, "register split");
static_assert(SG == 4, "scales are fetched four blocks at a time");
static_assert(P_SMEM <= 227 * 1024, "shared memory");

__device__ __forceinline__ void umma_f8_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 consecutive TMEM columns of this warp's 32 lanes; there after tmem_wait()
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Arrive on an accumulator's barrier of either CTA.  Relaxed: the sums are in registers (tcgen05.wait::ld) and
// nothing else is handed over; the releasing form waits for the warp's memory accesses at cluster scope
// every time (the membar stall then led all others, 8192 x 11008 x 4096 took 831 us, with relaxed arrivals 557).
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Every warp of both CTAs, before any of them leaves: the pair's MMAs are done and no arrival is on its way to
// the other CTA.  (Met from both sides of the register split, whose code must not join again.)
__device__ __forceinline__ void pair_exit_barrier() {
  __syncwarp();
  asm volatile("bar.sync 0, %0;" ::"n"(P_THREADS) : "memory");
  cluster_sync();
}

// shared -> global copy of a tile of a stack of matrices
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}

template <bool BLOCK, int VEC, typename TY>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P_THREADS, 1)
    fp8_matmul_pair_kernel(const __grid_constant__ CUtensorMap map_t, const __grid_constant__ CUtensorMap map_w,
                           const __grid_constant__ CUtensorMap map_y, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_tiles = smem + P_STAGES * P_STAGE_BYTES;
  float* staged = reinterpret_cast<float*>(out_tiles + P_OUT_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(out_tiles + P_OUT_BYTES + P_SCALE_BYTES);
  uint64_t* empty = full + P_STAGES;
  uint64_t* acc_full = empty + P_STAGES;  // [buffer][half]
  uint64_t* acc_empty = acc_full + 4;
  uint64_t* drain = acc_empty + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x / 32), 0), lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();  // 0 leads the pair
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < P_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);  // both issuers are through with the stage
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], P_EPI_WARPS);  // four warps of each CTA
    }
    mbar_init(drain, 2);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any arrival crosses the pair
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer (this CTA's halves)
      Ring<P_STAGES> r;
      uint32_t issued = 0;
      bool ok = true;
      const uint32_t full0 = mapa_shared(full, 0);  // the even CTA's stage barriers
      for (int u = pair; u < a.units && ok; u += n_pairs) {
        int tt, tw, s;
        unit_coords(u, a, tt, tw, s);
        const int b1 = min(a.kb, (s + 1) * a.kb_per_split);
        for (int b = s * a.kb_per_split; b < b1; ++b, ++issued, r.next()) {
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[r.slot], r.parity ^ 1, abort_flag, a.status, 61));
          if (!ok) break;
          if (elect_one()) {
            uint8_t* T = smem + r.slot * P_STAGE_BYTES;
            const uint32_t bar = full0 + r.slot * 8;
            if (rank == 0) mbar_expect_tx(&full[r.slot], 2 * P_STAGE_BYTES);
            tma_load_2d_pair(T, &map_t, b * BK, tt * 2 * BM + BM * (int)rank, bar);
            // of each half's 128 weight rows, this CTA's 64
            tma_load_2d_pair(T + BM * BK, &map_w, b * BK, tw * PN + 64 * (int)rank, bar);
            tma_load_2d_pair(T + BM * BK + 64 * BK, &map_w, b * BK, tw * PN + 128 + 64 * (int)rank, bar);
          }
          __syncwarp();
        }
      }
      // the copies already issued land before the CTA leaves: the even CTA watches both CTAs' on its stage
      // barriers, and the cluster barrier at the end keeps the odd CTA resident until then
      if (!ok && rank == 0) {
        const uint32_t first = issued > P_STAGES ? issued - P_STAGES : 0;
        for (uint32_t i = first; i < issued; ++i) mbar_wait_drain_cluster(&full[i % P_STAGES], (i / P_STAGES) & 1);
      }
    } else if (warp == 1 || warp == 2) {
      if (rank == 0) {
        // -------------------------------------------------------------- MMA issuers (even CTA), one per half
        const uint32_t h = warp - 1;
        Ring<P_STAGES> r;
        Ring<2> acc;
        bool ok = true;
        const uint64_t desc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t w_off = (uint64_t)((BM * BK + h * 64 * BK) >> 4);
        for (int u = pair; u < a.units && ok; u += n_pairs) {
          int tt, tw, s;
          unit_coords(u, a, tt, tw, s);
          const int nb = min(a.kb, (s + 1) * a.kb_per_split) - s * a.kb_per_split;
          for (int b = 0; b < nb; ++b, r.next(), acc.next()) {
            const uint32_t half = 2 * acc.slot + h;
            ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty[half], acc.parity ^ 1, abort_flag, a.status, 62) &&
                                             mbar_wait(&full[r.slot], r.parity, abort_flag, a.status, 63));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t td = desc0 + (uint64_t)((r.slot * P_STAGE_BYTES) >> 4);
#pragma unroll
              for (int kk = 0; kk < BK / 32; ++kk)
                umma_f8_pair(tmem_base + half * 128, td + (uint64_t)(kk * 2), td + w_off + (uint64_t)(kk * 2), a.idesc,
                             kk > 0 ? 1u : 0u);
              umma_commit_pair(&acc_full[half]);
              umma_commit_pair(&empty[r.slot]);
            }
            __syncwarp();
          }
        }
        // every MMA of the pair is complete before either CTA frees TMEM or leaves
        if (elect_one()) umma_commit_pair(drain);
        __syncwarp();
      }
      mbar_wait_drain(drain, 0);  // (the odd CTA waits for the pair's last MMAs too)
    }
    __syncwarp();
    tc_fence_before();
    pair_exit_barrier();
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc_pair(tmem_base, 512);
    }
  } else {
    // ---------------------------------------------------------------- epilogue (this CTA's tokens)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int quad = warp & 3;
    const int half = (warp - 4) >> 2;  // columns 128 * half .. of the tile
    const int et = threadIdx.x & 127;  // this thread among the half's 128
    const int r4 = lane >> 2, c4 = 2 * (lane & 3);
    const uint32_t acc_empty0 = mapa_shared(acc_empty, 0);
    uint8_t* out_tile = out_tiles + (warp - 4) * 4096;
    uint32_t group = 0;
    Ring<2> at;  // the accumulator of the block in hand
    bool ok = true;  // as in the single-CTA kernel: no warp leaves the walk, the named barrier needs all
    for (int u = pair; u < a.units; u += n_pairs) {
      int tt, tw, s;
      unit_coords(u, a, tt, tw, s);
      const int b0 = s * a.kb_per_split, b1 = min(a.kb, b0 + a.kb_per_split);
      const int t0 = tt * 2 * BM + BM * (int)rank, w0 = tw * PN + 128 * half;
      // scales staged P_SG blocks at a time, each half its own; BLOCK: the tokens' times the weight rows' one
      const float* tsc = a.a_scales + (int64_t)min(t0 + et, a.m - 1) * a.kb;
      const float* wsc = BLOCK ? a.b_scales + (int64_t)(min(w0, a.n - 1) >> 7) * a.kb
                               : a.b_scales + (int64_t)min(w0 + et, a.n - 1) * a.kb;
      float t_next[P_SG], w_next[P_SG];
      auto fetch = [&](int g0) {
        fetch_scales<VEC>(tsc, g0, a.kb, t_next);
        fetch_scales<VEC>(wsc, g0, a.kb, w_next);
      };
      fetch(b0);
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      uint32_t v[2][16];
      auto load = [&](int q) {
        const uint32_t taddr = tmem_base + ((uint32_t)(32 * quad) << 16) + (2 * at.slot + half) * 128 + 16 * q;
        if constexpr (BLOCK) {
          tmem_ld_rows(taddr, v[q & 1]);
        } else {
          tmem_ld<2>(taddr, v[q & 1]);
          tmem_ld<2>(taddr + (16u << 16), v[q & 1] + 8);
        }
      };
      auto begin_block = [&]() {
        if (ok) ok = mbar_wait(&acc_full[2 * at.slot + half], at.parity, abort_flag, a.status, 66);
        tc_fence_after();
        load(0);
      };
      begin_block();
      for (int g0 = b0; g0 < b1; g0 += P_SG, ++group) {
        float* sc = staged + (half * 2 + (group & 1)) * P_SG * P_SCALE_ROW;  // the other buffer may still be read
#pragma unroll
        for (int i = 0; i < P_SG; ++i) {
          sc[i * P_SCALE_ROW + et] = BLOCK ? t_next[i] * w_next[i] : t_next[i];
          if (!BLOCK) sc[i * P_SCALE_ROW + BM + et] = w_next[i];
        }
        fetch(g0 + P_SG);
        asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
        const int g1 = min(b1, g0 + P_SG);
        for (int b = g0; b < g1; ++b, sc += P_SCALE_ROW) {
          uint64_t rs[BLOCK ? 1 : 4];
#pragma unroll
          for (int i = 0; i < (BLOCK ? 1 : 4); ++i) {
            const uint32_t r = __float_as_uint(sc[BLOCK ? 32 * quad + lane : 32 * quad + r4 + 8 * i]);
            rs[i] = pack2(r, r);
          }
          const float* csc = sc + BM + c4;
          // loads from TMEM run one step ahead, across blocks
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            tmem_wait();
            if (q < 7) {
              load(q + 1);
            } else {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_relaxed(acc_empty0 + (2 * at.slot + half) * 8);
              at.next();
              if (b + 1 < b1) begin_block();
            }
            if constexpr (BLOCK) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                acc[8 * q + i] = fma2(pack2(v[q & 1][2 * i], v[q & 1][2 * i + 1]), rs[0], acc[8 * q + i]);
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint64_t cs = *reinterpret_cast<const uint64_t*>(csc + 8 * (2 * q + j));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint32_t* p = &v[q & 1][8 * (i >> 1) + 4 * j + 2 * (i & 1)];
                  acc[16 * i + 2 * q + j] = fma2(mul2(pack2(p[0], p[1]), cs), rs[BLOCK ? 0 : i], acc[16 * i + 2 * q + j]);
                }
              }
            }
          }
        }
      }
      if (!ok) continue;
      const int row0 = t0 + 32 * quad;
      int rr = r4, cc = c4;  // opaque: addresses computed here, not kept in registers through the blocks
      asm volatile("" : "+r"(rr), "+r"(cc));
      if (a.vec_y) {
        // through shared memory as 32 rows x 128 bytes (16-byte chunks swizzled by the row, as the copy
        // expects), then asynchronously to Y; what lies past Y's edges is not written.  Stores straight
        // from the registers were 16 bytes of 32 rows at a time and cost 160 of the 557 us that 8192 x 11008 x
        // 4096 took with them.
        constexpr int OC = 128 / (int)sizeof(TY);  // columns per tile
#pragma unroll
        for (int o = 0; o < 128 / OC; ++o) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          if constexpr (BLOCK) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              constexpr int V = 16 / (int)sizeof(TY);
              TY h[V];
#pragma unroll
              for (int i = 0; i < V; i += 2) {
                float v0, v1;
                unpack2(acc[(o * OC + c * V + i) / 2], v0, v1);
                h[i] = from_f32<TY>(v0), h[i + 1] = from_f32<TY>(v1);
              }
              *reinterpret_cast<uint4*>(out_tile + lane * 128 + ((c ^ (lane & 7)) << 4)) = *reinterpret_cast<uint4*>(h);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < OC / 8; ++j) {
                float v0, v1;
                unpack2(acc[16 * i + o * (OC / 8) + j], v0, v1);
                const int byte = (8 * j + cc) * (int)sizeof(TY);
                TY* y = reinterpret_cast<TY*>(out_tile + (rr + 8 * i) * 128 + ((byte >> 4 ^ rr) << 4) + (byte & 15));
                store_pair(y, v0, v1, 2, true);
              }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row0 < a.m && w0 + o * OC < a.n) {
            tma_store_3d(&map_y, w0 + o * OC, row0, s, out_tile);
            bulk_commit();
          }
        }
      } else if constexpr (BLOCK) {
        if (row0 + lane < a.m && w0 < a.n)
          store_row<128>(acc, static_cast<TY*>(a.Y) + (int64_t)(row0 + lane) * a.n + w0, a.n - w0);
      } else {
        const bool even = a.pair_y;  // rows start on pairs
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = row0 + rr + 8 * i, w = w0 + cc;
          if (tok >= a.m) continue;
          TY* y = static_cast<TY*>(a.Y) + (int64_t)tok * a.n + w;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float v0, v1;
            unpack2(acc[16 * i + j], v0, v1);
            const int left = a.n - w - 8 * j;
            store_pair(y + 8 * j, v0, v1, left, even && left > 1);
          }
        }
      }
    }
    if (lane == 0) bulk_wait<0>();  // the copies to Y are complete
    tc_fence_before();
    pair_exit_barrier();
  }
}

// ------------------------------------------------------------------------------------------------
// A few tokens (up to 8, or 16 with smaller weights).  The weights' bytes are all that counts, and a tile's way through
// tensor maps, TMEM and a second launch for split sums takes longer than reading them (1 x 4096 x 4096: 9.9 us, here
// 6.5, 2.6 TB/s with the launch in it; 1 x 12288 x 16384: 47 us, 4.3 TB/s).  Here a CTA takes 16 weight rows, its 8
// warps the blocks in turn; codes go straight from global memory into registers, two blocks ahead, become fp16 pairs
// (exact) and fragments of mma.m16n8k16 with the weights on the M side; the warps' scaled sums meet in shared
// memory, added in order.
// Every warp converts all tokens for itself, so with 9 to 16 of them large weights are better off in tiles: 16 x 768 x
// 768 2.6 us here, 4.8 in tiles, 4096 x 4096 8.4 and 10.8, 11008 x 4096 19.9 and 17.2, 12288 x 12288 52 and 39 (up to
// 8 tokens: 39 and 38).  With 32 the tiles win from 4096 x 4096 on (12.4 and 11.4).
bool few_tokens(int64_t m, int64_t n, int64_t k) { return m <= 8 || (m <= 16 && n * k <= 1 << 25); }
constexpr int kFewWarps = 8;
constexpr int kFewBlocks = 2;  // blocks a warp works on while as many are on their way

__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane holds columns 16 t .. 16 t + 15 of each half of a block, of weight rows g and g + 8 and of tokens g, g + 8, ..
// (NG of them); which columns meet in one MMA is free as long as both operands agree.
template <int NG, bool BLOCK, typename TY>
__global__ void __launch_bounds__(kFewWarps * 32, 2) fp8_matmul_few_kernel(const uint8_t* __restrict__ A,
                                                                           const float* __restrict__ a_scales,
                                                                           const uint8_t* __restrict__ B,
                                                                           const float* __restrict__ b_scales, int m,
                                                                           int n, int k, int kb, TY* __restrict__ Y) {
  __shared__ float sums[kFewWarps][16][8 * NG + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int row0 = blockIdx.x * 16;
  const int r0 = min(row0 + g, n - 1), r1 = min(row0 + g + 8, n - 1);
  const uint8_t* w0 = B + (int64_t)r0 * k + 16 * t;
  const uint8_t* w1 = B + (int64_t)r1 * k + 16 * t;
  const float* s0 = b_scales + (int64_t)(BLOCK ? r0 >> 7 : r0) * kb;
  const float* s1 = b_scales + (int64_t)(BLOCK ? r1 >> 7 : r1) * kb;
  const uint8_t* x[NG];
  const float *e0[NG], *e1[NG];
  float acc[NG][4];
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    x[n] = A + (int64_t)min(8 * n + g, m - 1) * k + 16 * t;  // past the last token: it once more, nobody reads the sums
    e0[n] = a_scales + (int64_t)min(8 * n + 2 * t, m - 1) * kb;
    e1[n] = a_scales + (int64_t)min(8 * n + 2 * t + 1, m - 1) * kb;
    acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 next[kFewBlocks][4];
  auto load = [&](int b0) {
#pragma unroll
    for (int i = 0; i < kFewBlocks; ++i) {
      const int c = (b0 + i * kFewWarps) * BK;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool ok = c + 64 * h + 16 * t < k;
        next[i][2 * h] = ok ? __ldg(reinterpret_cast<const uint4*>(w0 + c + 64 * h)) : zero;
        next[i][2 * h + 1] = ok ? __ldg(reinterpret_cast<const uint4*>(w1 + c + 64 * h)) : zero;
      }
    }
  };
  load(warp);
  for (int b0 = warp; b0 < kb; b0 += kFewWarps * kFewBlocks) {
    uint4 w[kFewBlocks][4];
#pragma unroll
    for (int i = 0; i < kFewBlocks; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i][j] = next[i][j];
    load(b0 + kFewWarps * kFewBlocks);
#pragma unroll
    for (int i = 0; i < kFewBlocks; ++i) {
      const int b = b0 + i * kFewWarps;
      if (b >= kb) break;
      float sum[NG][4];
#pragma unroll
      for (int n = 0; n < NG; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool ok = b * BK + 64 * h + 16 * t < k;
        uint4 xv[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) xv[n] = ok ? __ldg(reinterpret_cast<const uint4*>(x[n] + b * BK + 64 * h)) : zero;
        const uint4 u0 = w[i][2 * h], u1 = w[i][2 * h + 1];
        const uint32_t a0[4] = {u0.x, u0.y, u0.z, u0.w}, a1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t p0, p1, p2, p3, y0, y1;
          e4m3_to_f16(a0[q], p0, p2);
          e4m3_to_f16(a1[q], p1, p3);
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const uint32_t xw[4] = {xv[n].x, xv[n].y, xv[n].z, xv[n].w};
            e4m3_to_f16(xw[q], y0, y1);
            mma_f16(sum[n], p0, p1, p2, p3, y0, y1);
          }
        }
      }
      const float f0 = __ldg(s0 + b), f1 = __ldg(s1 + b);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const float c0 = __ldg(e0[n] + b), c1 = __ldg(e1[n] + b);
        acc[n][0] = fmaf(sum[n][0] * c0, f0, acc[n][0]);
        acc[n][1] = fmaf(sum[n][1] * c1, f0, acc[n][1]);
        acc[n][2] = fmaf(sum[n][2] * c0, f1, acc[n][2]);
        acc[n][3] = fmaf(sum[n][3] * c1, f1, acc[n][3]);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    sums[warp][g][8 * n + 2 * t] = acc[n][0], sums[warp][g][8 * n + 2 * t + 1] = acc[n][1];
    sums[warp][g + 8][8 * n + 2 * t] = acc[n][2], sums[warp][g + 8][8 * n + 2 * t + 1] = acc[n][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * m; i += kFewWarps * 32) {
    const int r = i & 15, tok = i >> 4;
    if (row0 + r < n) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) s += sums[w][r][tok];
      Y[(int64_t)tok * n + row0 + r] = from_f32<TY>(s);
    }
  }
}

template <typename TY>
gptq_status launch_few(const void* A, const float* a_scales, const void* B, const float* b_scales, bool block, int m,
                       int n, int k, TY* Y, cudaStream_t s) {
  const uint8_t *a = static_cast<const uint8_t*>(A), *b = static_cast<const uint8_t*>(B);
  const unsigned grid = (unsigned)((n + 15) / 16);
  const int kb = (k + BK - 1) / BK;
  auto kernel = m <= 8 ? (block ? fp8_matmul_few_kernel<1, true, TY> : fp8_matmul_few_kernel<1, false, TY>)
                       : (block ? fp8_matmul_few_kernel<2, true, TY> : fp8_matmul_few_kernel<2, false, TY>);
  kernel<<<grid, kFewWarps * 32, 0, s>>>(a, a_scales, b, b_scales, m, n, k, kb, Y);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

// Y = the splits' partial sums, added in split order; their rows are ld floats apart.
template <typename TY>
__global__ void __launch_bounds__(256) fp8_matmul_reduce_kernel(const float* __restrict__ partial, int splits, int m,
                                                                int n, int ld, TY* __restrict__ Y) {
  const int64_t plane = (int64_t)m * ld;
  for (int r = blockIdx.y; r < m; r += gridDim.y) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= n) continue;
    float s = 0.0f;
    for (int t = 0; t < splits; ++t) s += partial[t * plane + (int64_t)r * ld + c];
    Y[(int64_t)r * n + c] = from_f32<TY>(s);
  }
}

struct Plan {
  int nt, tiles_t, tiles_w, kb, kb_per_split, splits;  // nt = 256: the pair form
};

// Form, tile width and split of the blocks with the lowest estimated time in cycles, from times of single sizes: a
// block takes a CTA of the single form 480 + 3.6 NT (the epilogue's way through TMEM; NT = 32, 64, 128:
// 17 x 4096 x 4096 in 12.8, 15.7, 17.3 us; 96 where 128 leaves CTAs idle and 64 fills them twice: 333 x 4099 x 11008
// in 49.5 us without it, 44.5 with it) and a pair 1100 for four times the widest tile's area (1600 with a scale per
// weight row); a unit takes 2000 or 6000 for its fill and its end; split sums are written and read back at about
// 3000 bytes per cycle of the whole GPU, plus a launch.
Plan make_plan(int64_t m, int64_t n, int64_t k, bool block) {
  Plan best = {};
  double best_cost = 1e300;
  const int kb = (int)((k + BK - 1) / BK);
  auto consider = [&](int nt, int64_t tt, int64_t tw, int ctas, double block, double unit) {
    for (int want = 1; want <= 16 && want <= kb; ++want) {
      // splits start on multiples of 4 blocks so that their scales' 16-byte loads stay aligned
      const int per = want == 1 ? kb : ((kb + want - 1) / want + 3) / 4 * 4, splits = (kb + per - 1) / per;
      if (splits != want) continue;
      const int64_t units = tt * tw * splits;
      if (splits > 1 && units > 2 * kPlanSMs / ctas) continue;
      const double waves = (double)((units + kPlanSMs / ctas - 1) / (kPlanSMs / ctas));
      double cost = waves * (per * block + unit);
      if (splits > 1) cost += 8.0 * splits * (double)m * (double)n / 3000.0 + 5700.0;
      if (cost < best_cost) {
        best_cost = cost;
        best = {nt, (int)tt, (int)tw, kb, per, splits};
      }
    }
  };
  for (int nt = 32; nt <= 128; nt += 32)
    if (nt != 96 || !block)  // 128 weight rows that share a scale do not divide into 96
      consider(nt, (m + BM - 1) / BM, (n + nt - 1) / nt, 1, 480.0 + 3.6 * nt, 2000.0);
  if (m > BM) consider(PN, (m + 2 * BM - 1) / (2 * BM), (n + PN - 1) / PN, 2, block ? 1100.0 : 1600.0, 6000.0);
  return best;
}

// the split sums' row stride: rows on 16 bytes, as the pair form's copies need them
int64_t partial_stride(int64_t n) { return (n + 3) / 4 * 4; }

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

// Y, or the split sums as a stack of matrices, in tiles of 32 rows x 128 bytes with the 128-byte swizzle
template <typename TY>
bool out_map(CUtensorMap* map, void* base, int64_t m, int64_t n, int64_t ld, int64_t stack) {
  auto encode = encode_fn();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)n, (cuuint64_t)m, (cuuint64_t)stack};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * sizeof(TY)), (cuuint64_t)(m * ld * sizeof(TY))};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / sizeof(TY)), 32, 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUtensorMapDataType type = std::is_same<TY, float>::value    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : std::is_same<TY, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return encode(map, type, 3, base, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int NT, bool BLOCK, typename TY>
gptq_status launch(const CUtensorMap& t, const CUtensorMap& w, Args a, int sms, cudaStream_t s) {
  auto kernel = a.scale_width == 4   ? fp8_matmul_kernel<NT, BLOCK, 4, TY>
                : a.scale_width == 2 ? fp8_matmul_kernel<NT, BLOCK, 2, TY>
                                     : fp8_matmul_kernel<NT, BLOCK, 1, TY>;
  // D fp32 (bit 4), A and B e4m3 (0), both K-major, N = NT, M = 128
  a.idesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
  GPTQ_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NT>::kSmem));
  kernel<<<std::min(a.units, sms), Cfg<NT>::kThreads, Cfg<NT>::kSmem, s>>>(t, w, a);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <bool BLOCK, typename TY>
gptq_status launch_pair(const CUtensorMap& t, const CUtensorMap& w, Args a, int sms, cudaStream_t s) {
  CUtensorMap y = t;  // not used unless Y's rows are aligned
  if (a.vec_y && !out_map<TY>(&y, a.Y, a.m, a.n, a.partial ? a.ld : a.n, a.splits)) return GPTQ_ERR_CUDA;
  auto kernel = a.scale_width == 4   ? fp8_matmul_pair_kernel<BLOCK, 4, TY>
                : a.scale_width == 2 ? fp8_matmul_pair_kernel<BLOCK, 2, TY>
                                     : fp8_matmul_pair_kernel<BLOCK, 1, TY>;
  a.idesc = (1u << 4) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)((2 * BM) >> 4) << 24);
  cudaFuncAttributes attr;  // the register split draws on the launch's registers: never ask for more than those
  GPTQ_CUDA_TRY(cudaFuncGetAttributes(&attr, kernel));
  if (attr.numRegs < kLaunchRegs) return GPTQ_ERR_CUDA;
  GPTQ_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P_SMEM));
  kernel<<<2 * std::min(a.units, sms / 2), P_THREADS, P_SMEM, s>>>(t, w, y, a);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <int NT, typename TY>
gptq_status launch_block(bool block, const CUtensorMap& t, const CUtensorMap& w, const Args& a, int sms,
                         cudaStream_t s) {
  return block ? launch<NT, true, TY>(t, w, a, sms, s) : launch<NT, false, TY>(t, w, a, sms, s);
}

template <typename TY>
gptq_status launch_typed(const Plan& p, bool block, const CUtensorMap& t, const CUtensorMap& w, const Args& a, int sms,
                         cudaStream_t s) {
  gptq_status st;
  switch (p.nt) {
    case 32: st = launch_block<32, TY>(block, t, w, a, sms, s); break;
    case 64: st = launch_block<64, TY>(block, t, w, a, sms, s); break;
    case 96: st = launch<96, false, TY>(t, w, a, sms, s); break;  // never with block scales
    case 128: st = launch_block<128, TY>(block, t, w, a, sms, s); break;
    default: {
      if (a.partial == nullptr) {
        st = block ? launch_pair<true, TY>(t, w, a, sms, s) : launch_pair<false, TY>(t, w, a, sms, s);
      } else {  // split sums: fp32, in rows that the copies can write
        Args b = a;
        b.Y = a.partial, b.vec_y = true;
        st = block ? launch_pair<true, float>(t, w, b, sms, s) : launch_pair<false, float>(t, w, b, sms, s);
      }
    }
  }
  if (st != GPTQ_OK || a.partial == nullptr) return st;
  const dim3 grid((unsigned)((a.n + 255) / 256), (unsigned)std::min(a.m, 1024));
  fp8_matmul_reduce_kernel<TY><<<grid, 256, 0, s>>>(a.partial, a.splits, a.m, a.n, a.ld, static_cast<TY*>(a.Y));
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace


size_t fp8_matmul_workspace(int64_t m, int64_t n, int64_t k) {
  if (few_tokens(m, n, k)) return 0;
  size_t need = 0;  // for either kind of weight scales
  for (int block = 0; block < 2; ++block) {
    const Plan p = make_plan(m, n, k, block != 0);
    if (p.splits > 1) need = std::max(need, align_up((size_t)p.splits * m * partial_stride(n) * sizeof(float), 256));
  }
  return need;
}

gptq_status fp8_matmul_launch(const void* A, const float* a_scales, const void* B, const float* b_scales,
                              int32_t b_block_rows, int64_t m, int64_t n, int64_t k, void* Y, int32_t y_dtype,
                              int32_t* status, void* workspace, cudaStream_t stream) {
  if (few_tokens(m, n, k)) {
    const bool block = b_block_rows == 128;
    switch (y_dtype) {
      case GPTQ_BF16: return launch_few(A, a_scales, B, b_scales, block, (int)m, (int)n, (int)k, static_cast<__nv_bfloat16*>(Y), stream);
      case GPTQ_FP16: return launch_few(A, a_scales, B, b_scales, block, (int)m, (int)n, (int)k, static_cast<__half*>(Y), stream);
      default: return launch_few(A, a_scales, B, b_scales, block, (int)m, (int)n, (int)k, static_cast<float*>(Y), stream);
    }
  }
  const Plan p = make_plan(m, n, k, b_block_rows == 128);
  const int64_t units = (int64_t)p.tiles_w * p.tiles_t * p.splits;
  if (units > 0x7fffffff - kPlanSMs) return GPTQ_ERR_ARG;
  const int token_rows = (int)std::min<int64_t>(BM, (m + 7) / 8 * 8);  // whole swizzle atoms of 8 rows
  CUtensorMap t, w;
  if (!operand_map(&t, A, m, k, token_rows) || !operand_map(&w, B, n, k, p.nt == PN ? 64 : p.nt)) return GPTQ_ERR_CUDA;
  int dev = 0, sms = 0;
  GPTQ_CUDA_TRY(cudaGetDevice(&dev));
  GPTQ_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  Args a = {};
  a.m = (int)m, a.n = (int)n, a.kb = p.kb;
  a.tiles_w = p.tiles_w, a.tiles_t = p.tiles_t, a.units = (int)units;
  a.kb_per_split = p.kb_per_split;
  a.token_bytes = token_rows * BK;
  a.scale_width = 4;
  while (a.scale_width > 1 && (p.kb % a.scale_width || !aligned(a_scales, 4 * a.scale_width) ||
                               !aligned(b_scales, 4 * a.scale_width)))
    a.scale_width /= 2;
  const int y_size = y_dtype == GPTQ_FP32 ? 4 : 2;
  a.vec_y = n * y_size % 16 == 0 && aligned(Y, 16);
  a.pair_y = n % 2 == 0 && aligned(Y, 2 * y_size);
  const bool block = b_block_rows == 128;
  a.a_scales = a_scales, a.b_scales = b_scales;
  a.Y = Y;
  a.partial = p.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  a.ld = (int)partial_stride(n), a.splits = p.splits;
  a.status = status;
  switch (y_dtype) {
    case GPTQ_BF16: return launch_typed<__nv_bfloat16>(p, block, t, w, a, sms, stream);
    case GPTQ_FP16: return launch_typed<__half>(p, block, t, w, a, sms, stream);
    default: return launch_typed<float>(p, block, t, w, a, sms, stream);
  }
}

}  // namespace gptq
