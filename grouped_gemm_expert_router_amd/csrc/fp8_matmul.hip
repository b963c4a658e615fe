// Dense products of blockwise e4m3 operands on gfx950's fp8 MFMA (v_mfma_scale_f32_32x32x64_f8f6f4 with
// unit block exponents): C = A . B (+ C_in) with one scale per row and 128 values of K for A, and for B
// one per 128 x 128 block or one per row and 128 values.  Blockwise FP8 is one of the data types of the
// fused MoE backward on the Prime Mega MoE page ("Prime Mega MoE: tanításra is jó a DeepSeek MoE
// kernele", section "Mit csinált a Prime Intellect?").
#include <type_traits>

#include "common.hpp"
#include "gemm_common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// N-contiguous operand tile of 128 columns in LDS: [k][128 bytes], chunk c (16 columns) of k row r at
// chunk c ^ (2 * ((r >> 1) & 3)): the 8 rows x 32 columns that an LDS cycle serves hit all banks.
__device__ __forceinline__ uint32_t kn8n_off(int kr, int col) {
  return kr * 128 + ((((col >> 4) ^ (2 * ((kr >> 1) & 3)))) << 4) + (col & 15);
}
__device__ __forceinline__ i32x8 read_kn8n(uint32_t base, int cbase, int kk, int lane) {
  const int grp = lane >> 4, i16 = lane & 15;
  const int col = cbase + 16 * (grp & 1) + 8 * (i16 & 1);
  const int krb = 64 * kk + 32 * (grp >> 1) + (i16 >> 1);
  i32x8 v;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const i32x2v t = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS_AS i32x2v*)(uintptr_t)(base + kn8n_off(krb + 8 * h, col)));
    v[2 * h] = t.x;
    v[2 * h + 1] = t.y;
  }
  return v;
}

// Codes 8s .. 8s+7 of a lane's 32 as bf16, exactly.
__device__ __forceinline__ bf16x8_t widened(const i32x8& v, int s) {
  bf16x8_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2_t p = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * s + i / 2], 1.0f, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * s + i / 2], 1.0f, false);
    w[2 * i] = p[0];
    w[2 * i + 1] = p[1];
  }
  return w;
}

// The products of two 32 x 64 fragments added to c (B first: the block of C is transposed).
//
// A bf16 C takes the fp8 instruction, 4.1 PFLOP/s where the bf16 one has 1.65.  That instruction adds
// products eight at a time (k = 8i .. 8i+7), aligned to the largest of the eight, and drops what lies
// more than 13 bits below it (measured: 2^16 + 2^2 in one group is 2^16, in two groups exact): at most
// 7 2^-13 of the eight products' magnitudes, 1.5e-5 of the result's norm on normal data, a hundredth of
// C's own rounding.  An fp32 C keeps the codes' products whole: e4m3 values are bf16 values, and the bf16
// instruction rounds as fp32 does.
template <bool WHOLE>
__device__ __forceinline__ f32x16_t multiply(const i32x8& b, const i32x8& a, f32x16_t c) {
  if constexpr (WHOLE) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widened(b, s), widened(a, s), c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 0, 0, 0, 127, 0, 127);
  }
}

// The same of two 16 x 128 fragments: lane l holds row l % 16 and the codes of its quarter l / 16 of K.
template <bool WHOLE>
__device__ __forceinline__ f32x4_t multiply16(const i32x8& b, const i32x8& a) {
  f32x4_t c = {};
  if constexpr (WHOLE) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widened(b, s), widened(a, s), c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, 0, 127, 0, 127);
  }
}

// Four neighbouring values of C from its value `at` on, with C_in.
template <bool F32>
__device__ __forceinline__ void store4(const MatmulArgs& g, int64_t at, float (&v)[4]) {
  if (g.C_in) {
    if constexpr (F32) {
      const float4 a = *(const float4*)((const float*)g.C_in + at);
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    } else {
      const u32x2 a = *(const u32x2*)((const uint16_t*)g.C_in + at);
      v[0] += lo_bf16(a.x), v[1] += hi_bf16(a.x), v[2] += lo_bf16(a.y), v[3] += hi_bf16(a.y);
    }
  }
  if constexpr (F32) *(float4*)((float*)g.C + at) = make_float4(v[0], v[1], v[2], v[3]);
  else *(u32x2*)((uint16_t*)g.C + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

}  // namespace

// ------------------------------------------------------------------------------------ few rows
// The product of few rows is a reading of B.  A wave takes whole blocks of K (128 deep) of a few columns, its own
// ones, so that no wave waits for another until the end: B by DMA into LDS of the wave's own, whole cache
// lines a row (a load that takes 64 bytes of 16 rows ran at half the rate).  Up to 16 rows of A go into registers
// from L2; more of them through the wave's LDS as well (48x7168x2048: 8.5 us, from L2 into registers 15.5).  The
// waves' sums meet in LDS in a fixed order; where the columns alone give too few thread blocks, K is cut once
// more over `splits` of them, whose fp32 sums fp8_matmul_sum_kernel adds in order.
//
// B [N, K]: 16 columns a thread block, whose eight waves take the blocks of K in turn, U at a time.
// B [K, N]: 16 NF columns, 128 (one cache line) where K is long; the LDS transpose read makes the operands.
// 1x4096x7168: 8.4 us (3.5 TB/s of B) and 2.5 for the sum, 11.0 the call; a plain read of as many bytes takes 5.4.
template <bool KN, bool ROWS, bool WHOLE, int MF, int NF, int U>
__global__ __launch_bounds__(512) void fp8_matmul_few_kernel(const MatmulArgs g, float* __restrict__ part,
                                                                        int per) {
  constexpr int KW = 8;                // waves, which share K
  constexpr bool AL = MF > 1;          // A by way of LDS too
  constexpr int B_BLK = 2048 * NF, BLK = B_BLK + (AL ? 2048 * MF : 0);  // bytes of a block of K
  static_assert(!KN || !ROWS, "");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[8 * U * BLK];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)xcd_remap(blockIdx.x, gridDim.x) * (16 * NF);
  const int KB = (int)((g.K + 127) / 128);
  const int64_t NB = (g.N + 127) / 128;
  const int kb0 = blockIdx.y * per, kb1 = min(KB, kb0 + per);
  const uint32_t mine = __builtin_amdgcn_readfirstlane(lds_addr_of(smem)) + wave * (U * BLK);
  const uint8_t* a_row[MF];
  const float* a_scale[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int64_t m = min((int64_t)(16 * i + l16), g.M - 1);  // rows past the last feed unstored values
    a_row[i] = g.A + m * g.lda;
    a_scale[i] = g.A_scale + m * KB;
  }
  f32x4_t acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = f32x4_t{};

  // One 1 KB DMA: eight rows of 128 bytes, lane l the piece l % 8 (swizzled) of row l / 8.  What lies past
  // K or N comes from the operand's own last rows or columns, so that no address leaves it; past K, A's
  // pieces are zeros and B's are cleared in the operands.
  auto issue = [&](int kb, int u) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)kb * 128;
#pragma unroll
    for (int j = 0; j < 2 * NF; ++j) {
      const uint8_t* src;
      if constexpr (KN) {
        const int r = (64 * j + lane) / NF, c = NF == 8 ? (lane & 7) ^ (2 * ((r >> 1) & 3)) : lane % NF;
        src = g.B + min(k0 + r, g.K - 1) * g.ldb + min(n0 + 16 * c, g.N - 16);
      } else {
        const int r = 8 * j + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
        src = g.B + min(n0 + r, g.N - 1) * g.ldb + min(k0 + 16 * c, g.K - 16);
      }
      dma16(src, mine + u * BLK + 1024 * j);
    }
    if constexpr (AL) {
#pragma unroll
      for (int j = 0; j < 2 * MF; ++j) {
        const int r = 8 * j + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
        dma16(g.A + min((int64_t)r, g.M - 1) * g.lda + min(k0 + 16 * c, g.K - 16), mine + u * BLK + B_BLK + 1024 * j);
      }
    }
  };
  struct Row {
    i32x8 a[AL ? 1 : MF];
    float sa[MF], sb[ROWS ? 4 * NF : KN ? 1 : NF];
  };
  // the 32 bytes of K that lane l has of its row: 16-byte pieces q and q + 4 of the block
  auto load = [&](Row& c, int kb) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)kb * 128 + 16 * q;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      if constexpr (!AL) {
        u32x4 lo = {}, hi = {};
        if (k0 < g.K) lo = *(const u32x4*)(a_row[i] + k0);
        if (k0 + 64 < g.K) hi = *(const u32x4*)(a_row[i] + k0 + 64);
        c.a[i] = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
      }
      c.sa[i] = a_scale[i][kb];
    }
    if constexpr (KN) {
      c.sb[0] = g.B_scale[kb * NB + min(n0 / 128, NB - 1)];
    } else {
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const int64_t n = min(n0 + 16 * j, g.N - 16);
        if constexpr (ROWS) {
#pragma unroll
          for (int r = 0; r < 4; ++r) c.sb[4 * j + r] = g.B_scale[(n + 4 * q + r) * KB + kb];
        } else {
          c.sb[j] = g.B_scale[n / 128 * KB + kb];
        }
      }
    }
  };
  auto add = [&](const Row& c, int kb, int u) __attribute__((always_inline)) {
    const uint32_t base = mine + u * BLK;
    const int64_t left = g.K - (int64_t)kb * 128 - 16 * q;  // codes of K from the lane's first on
    auto pieces = [&](uint32_t at, int row) __attribute__((always_inline)) {
      const u32x4 lo = *(const LDS_AS u32x4*)(uintptr_t)(at + km_off<64>(row, q));
      const u32x4 hi = *(const LDS_AS u32x4*)(uintptr_t)(at + km_off<64>(row, q + 4));
      return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    // the last block: a NaN code would outlive the other operand's zero
    auto clear = [&](i32x8& v) __attribute__((always_inline)) {
#pragma unroll
      for (int w = 0; w < 8; ++w)
        if (left <= 64 * (w >> 2)) v[w] = 0;
    };
    i32x8 a[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      if constexpr (AL) {
        a[i] = pieces(base + B_BLK, 16 * i + l16);
        clear(a[i]);
      } else {
        a[i] = c.a[i];
      }
    }
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      i32x8 b;
      if constexpr (KN) {
        // of a group of 16 lanes, lane s addresses 8 columns of row s / 2 and gets 8 rows of column s
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int r = 16 * q + 8 * (h & 1) + 64 * (h >> 1) + (l16 >> 1);
          const i32x2v t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (LDS_AS i32x2v*)(uintptr_t)(base + (NF == 8 ? kn8n_off(r, 16 * j + 8 * (l16 & 1))
                                                          : r * (16 * NF) + 16 * j + 8 * (l16 & 1))));
          b[2 * h] = t.x;
          b[2 * h + 1] = t.y;
        }
      } else {
        b = pieces(base, 16 * j + l16);
      }
      clear(b);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const f32x4_t t = multiply16<WHOLE>(b, a[i]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(t[r], c.sa[i] * c.sb[ROWS ? 4 * j + r : KN ? 0 : j], acc[i][j][r]);
      }
    }
  };
  for (int kb = kb0 + wave; kb < kb1; kb += KW * U) {
    lds_wait();  // the wave's reads of what it now overwrites
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kb + KW * u < kb1) issue(kb + KW * u, u);
    Row c[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kb + KW * u < kb1) load(c[u], kb + KW * u);
    vm_wait<0>();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kb + KW * u < kb1) add(c[u], kb + KW * u, u);
  }
  // Lane l holds columns 4q .. 4q+3 of row l % 16 of each 16 x 16 piece.  Sixteen rows at a time.
  float4* red = (float4*)smem;
  constexpr int UNITS = NF * 64;
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NF; ++j)
      red[(wave * NF + j) * 64 + lane] = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
    __syncthreads();
    for (int u = threadIdx.x; u < UNITS; u += 512) {
      float v[4] = {};
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const float4 a = red[k * UNITS + u];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
      }
      const int64_t m = 16 * i + (u & 15), n = n0 + 16 * (u >> 6) + 4 * ((u & 63) >> 4);
      if (m >= g.M || n >= g.N) continue;
      if (part) *(float4*)(part + ((int64_t)blockIdx.y * g.M + m) * g.N + n) = make_float4(v[0], v[1], v[2], v[3]);
      else store4<WHOLE>(g, m * g.ldc + n, v);
    }
  }
}

// What was cut along K: the tiles from `first` on, each held `splits` times as [bm][bn] in fp32.
struct Cut {
  int64_t first, tiles;  // the tile number the cut ones start at; how many there are
  int splits, per;       // parts; blocks of K a part
  int64_t bm, bn;
  int nM, nN, gm;
};

// The sums of the parts of K, in order; four values a thread.
template <bool F32>
__global__ __launch_bounds__(256) void fp8_matmul_sum_kernel(const MatmulArgs g, const float* __restrict__ part, const Cut cut) {
  const int64_t u = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, size = cut.bm * cut.bn, tile = u / size;
  if (tile >= cut.tiles) return;
  const int2 at = grouped_tile((int)(cut.first + tile), cut.nM, cut.nN, cut.gm);
  const int64_t r = (u - tile * size) / cut.bn, c = u - tile * size - r * cut.bn;
  const int64_t m = at.x * cut.bm + r, n = at.y * cut.bn + c;
  if (m >= g.M || n >= g.N) return;
  float v[4] = {};
  for (int s0 = 0; s0 < cut.splits; s0 += 8) {  // eight loads in flight
    float4 a[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) a[s] = *(const float4*)(part + min(s0 + s, cut.splits - 1) * cut.tiles * size + u);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s0 + s < cut.splits) v[0] += a[s].x, v[1] += a[s].y, v[2] += a[s].z, v[3] += a[s].w;
  }
  store4<F32>(g, m * g.ldc + n, v);
}

// -------------------------------------------------------------------------------------- tiles
// What a tile kernel reads in the place of codes past K.
__device__ const uint4 g_zero = {0, 0, 0, 0};

// LDS DMA of 16 or 4 bytes a lane from a wave's base address and a lane's 32-bit offset.
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds_byte_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds_byte_addr)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds_byte_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds_byte_addr)
               : "memory", "m0");
}

template <typename T>
__device__ __forceinline__ const T* uniform_ptr(const T* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const T*)((uint64_t)lo | (uint64_t)hi << 32);
}

// BM x BN tiles, WM x WN waves, a block of K (128 deep) a step through S LDS stages, all by DMA.
//
// A step's DMAs go out one by one between the matrix instructions: issued together at the step's start
// they held every wave up for a third of the step (21804x4096x7168 790 us).
//
// Scales.  A row's scales lie along K, so the 4 bytes a step needs of a row come with a cache line of
// their own.  They are therefore fetched for eight blocks of K at a time, in the steps before they are
// used: one DMA brings one block's scales of 64 rows, and the waves of a step take the same rows for
// different blocks, and with them the same lines.
//
// Waves that have their fragments run at a higher priority (s_setprio) until their matrix instructions are out, so
// that those of a compute unit take turns between LDS and the matrix cores (1023x7168x4096 42.4 -> 41.0 us, with
// fp32 C 66.9 -> 64.3, 7168x4096x21808 with fp32 C 1335 -> 1263, all on one card; on others the last takes 1330 to
// 1380).  Counters at 4096x4096x7168: matrix cores busy 50 % of the time (21804x4096x7168 47 %, fp32 C 45 %), vector ALU
// (promotion, addresses) 39 %, LDS without conflicts; the rest is the barrier each step and the fragments that every
// wave reads behind it.  A second barrier inside the step, to send B's next block earlier,
// gave nothing.
//
// Each 32 x 32 block of C is held transposed (B is the MFMA's first operand): lane l has row l % 32 and 16
// columns, so one A scale serves its 16 values.
template <int FORM, bool WHOLE, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN, 1) void fp8_matmul_tile_kernel(const MatmulArgs g, float* __restrict__ part,
                                                                          const Cut cut) {
  constexpr bool KN = FORM == MOE_B_KN, ROWS = FORM == MOE_B_NK_ROWS;
  constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32, BK = 128;
  constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
  constexpr int QA = A_BYTES / 1024 / NW, QB = B_BYTES / 1024 / NW, NDMA = QA + QB;
  constexpr int NG = (BM + (ROWS ? BN : 0)) / 64;       // groups of 64 rows with scales
  constexpr int NBT = BN / 128;                         // B tiles with a scale
  constexpr int SC = 8 * 64 * NG * 4, SB = ROWS ? 0 : 8 * NBT * 4;  // bytes for eight blocks of K
  constexpr int NSC = S > 2 ? 3 : 2;                    // how many eights there are
  static_assert(QA * 1024 * NW == A_BYTES && QB * 1024 * NW == B_BYTES, "DMA split");
  static_assert(FN == 2 && BM % 64 == 0 && (!KN || BN == 128 || BN == 256), "layouts");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE + NSC * (SC + SB)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr_of(smem)), sc0 = lds0 + S * STAGE, sb0 = sc0 + NSC * SC;
  const int KB = (int)((g.K + 127) / 128), NB = (int)((g.N + 127) / 128);
  // tiles whole along K, then those that are cut
  const bool whole_tile = (int64_t)blockIdx.x < cut.first;
  const int nth = whole_tile ? xcd_remap(blockIdx.x, (int)cut.first)
                             : xcd_remap(blockIdx.x - (int)cut.first, gridDim.x - (int)cut.first);
  const int of_tile = whole_tile ? nth : nth / cut.splits, of_k = whole_tile ? 0 : nth - of_tile * cut.splits;
  const int kb0 = whole_tile ? 0 : of_k * cut.per, nk = whole_tile ? KB : min(KB - kb0, cut.per);
  const int2 tile = grouped_tile(whole_tile ? of_tile : (int)cut.first + of_tile, cut.nM, cut.nN, cut.gm);
  const int64_t m0 = (int64_t)tile.x * BM, n0 = (int64_t)tile.y * BN;
  const int mrows = (int)min((int64_t)BM, g.M - m0), ncols = (int)min((int64_t)BN, g.N - n0);

  // ------------------------------------------------------------------ DMA sources
  // DMA q of a wave: eight rows of 128 bytes (a [K, N] operand: 1024 / BN rows of BN bytes).  Rows and columns
  // past the tile's last are the last one again; they feed values that are not stored.
  auto a_row = [&](int q) __attribute__((always_inline)) { return min(8 * (wave * QA + q), mrows - 1); };
  auto b_row = [&](int q) __attribute__((always_inline)) {
    return KN ? 1024 / BN * (wave * QB + q) : min(8 * (wave * QB + q), ncols - 1);
  };
  // A lane's offset from its DMA's first row: the row's, at most that of the tile's last row, and the piece's.
  // Which piece a lane takes (the swizzle) depends on the DMA's parity alone.
  constexpr int BR = KN ? BN / 16 : 8;  // lanes a row of B
  const uint32_t a_lane = (uint32_t)(lane / 8) * (uint32_t)g.lda, b_lane = (uint32_t)(lane / BR) * (uint32_t)g.ldb;
  uint32_t piece[2], b_piece[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    piece[p] = 16 * ((lane % 8) ^ ((4 * p + lane / 16) & 7));
    const int kr = (1024 / BN * p + lane / BR) & 7;
    b_piece[p] = KN ? min(16 * (BN == 256 ? (lane % BR) ^ (2 * (kr & 7)) : (lane % BR) ^ (2 * ((kr >> 1) & 3))), ncols - 16)
                    : piece[p];
  }
  auto a_off = [&](int q) __attribute__((always_inline)) {
    return min(a_lane, (uint32_t)min(mrows - 1 - a_row(q), 7) * (uint32_t)g.lda) + piece[q & 1];
  };
  auto b_off = [&](int q) __attribute__((always_inline)) {
    const uint32_t p = b_piece[q & 1];
    return KN ? b_lane + p : min(b_lane, (uint32_t)min(ncols - 1 - b_row(q), 7) * (uint32_t)g.ldb) + p;
  };
  static_assert(QA % 2 == 0 && QB % 2 == 0, "a DMA's parity is its number's, the same in every wave");
  const uint8_t* a_base = uniform_ptr(g.A + m0 * g.lda + (int64_t)kb0 * BK);
  const uint8_t* b_base = uniform_ptr(KN ? g.B + (int64_t)kb0 * BK * g.ldb + n0 : g.B + n0 * g.ldb + (int64_t)kb0 * BK);
  const int64_t b_step = KN ? BK * g.ldb : BK;
  // DMA n of stage t
  auto dma = [&](int n, int t) __attribute__((always_inline)) {
    const uint32_t at = lds0 + t % S * STAGE;
    if (n < QA) dma16(a_base + (int64_t)t * BK + a_row(n) * g.lda, a_off(n), at + (wave * QA + n) * 1024);
    else dma16(b_base + t * b_step + b_row(n - QA) * g.ldb, b_off(n - QA), at + A_BYTES + (wave * QB + n - QA) * 1024);
  };
  // the last stage where it is a partial block: zeros past K
  auto dma_ragged = [&](int t) __attribute__((always_inline)) {
    const uint32_t at = lds0 + t % S * STAGE;
    const int left = (int)(g.K - (int64_t)(KB - 1) * BK);
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const int row = 8 * (wave * QA + q) + lane / 8, k = 16 * ((lane % 8) ^ ((row >> 1) & 7));
      const uint8_t* src = a_base + (int64_t)t * BK + a_row(q) * g.lda + a_off(q);
      dma16(k < left ? (const void*)src : (const void*)&g_zero, at + (wave * QA + q) * 1024);
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const int row = 8 * (wave * QB + q) + lane / 8;
      const int k = KN ? b_row(q) + lane / (BN / 16) : 16 * ((lane % 8) ^ ((row >> 1) & 7));
      const uint8_t* src = b_base + t * b_step + b_row(q) * g.ldb + b_off(q);
      dma16(k < left ? (const void*)src : (const void*)&g_zero, at + A_BYTES + (wave * QB + q) * 1024);
    }
  };
  const bool ragged = g.K % BK != 0 && kb0 + nk == KB;
  const float* sa_base = uniform_ptr(g.A_scale + m0 * KB);
  const float* sb_base = uniform_ptr(ROWS ? g.B_scale + n0 * KB : g.B_scale + n0 / 128 * (KN ? 1 : KB));
  // the scales of unit `id` of the eight blocks from the thread block's block k8 on: block id % 8, group id / 8
  auto scales = [&](int k8, int id) __attribute__((always_inline)) {
    const int k = id & 7, grp = id >> 3, kb = min(kb0 + k8 + k, KB - 1);
    const bool of_b = ROWS && grp >= BM / 64;
    const int row = of_b ? min(64 * (grp - BM / 64) + lane, ncols - 1) : min(64 * grp + lane, mrows - 1);
    dma4(of_b ? sb_base : sa_base, 4u * (uint32_t)(row * KB + kb), sc0 + (k8 >> 3) % NSC * SC + (k * NG + grp) * 256);
  };
  auto b_tile_scales = [&](int k8) __attribute__((always_inline)) {
    if constexpr (!ROWS) {
      const int first = min(kb0 + k8, KB - 1), k = min(lane / NBT, KB - 1 - first);
      const int nb = min(lane % NBT, (ncols + 127) / 128 - 1);
      if (lane < 8 * NBT)
        dma4(sb_base + (int64_t)first * (KN ? NB : 1), 4u * (uint32_t)(KN ? k * NB + nb : nb * KB + k),
             sb0 + (k8 >> 3) % NSC * SB);
    }
  };
  // the wave's share, in step t, of the scales of the eight blocks behind block t's eight
  auto step_scales = [&](int t) __attribute__((always_inline)) {
    static_assert(NG <= NW, "a wave has at most one unit a step");
    const int id = (t & 7) * NW + wave;
    if (id < 8 * NG) scales((t & ~7) + 8, id);
    if ((t & 7) == 7 && wave == NW - 1) b_tile_scales((t & ~7) + 8);
  };

  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x16_t{};

  // Step t, with the DMAs of stage t + S - 1 between its matrix instructions where MORE.  (No branch decides
  // on a DMA: the compiler would move the matrix instructions past it.)
  auto compute = [&](int t, auto more) __attribute__((always_inline)) {
    constexpr bool MORE = decltype(more)::value;
    const uint32_t abase = lds0 + t % S * STAGE, bbase = abase + A_BYTES;
    const uint32_t sbase = sc0 + (t >> 3) % NSC * SC + (t & 7) * NG * 256;
    auto b_frag = [&](int j, int kk) __attribute__((always_inline)) -> i32x8 {
      const int col = wn * TN + 32 * j;
      if constexpr (KN && BN == 256) return read_kn8(bbase, col, kk, lane);
      else if constexpr (KN) return read_kn8n(bbase, col, kk, lane);
      else return read_km8(bbase, col + (lane & 31), kk, lane);
    };
    auto a_frag = [&](int i, int kk) __attribute__((always_inline)) {
      return read_km8(abase, wm * TM + 32 * i + (lane & 31), kk, lane);
    };
    auto fence = [] __attribute__((always_inline)) { __builtin_amdgcn_sched_barrier(0); };
    int sent = 0;  // a constant at every place, once unrolled
    auto send = [&](int n) __attribute__((always_inline)) {
      if constexpr (MORE)
#pragma unroll
        for (int u = 0; u < n; ++u, ++sent)
          if (sent < NDMA) dma(sent, t + S - 1);
    };
    auto promote = [&](int i, int j, const f32x16_t& c, const float (&sa)[FM], float sb) __attribute__((always_inline)) {
      if constexpr (ROWS) {
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const f32x4_t s4 = *(const LDS_AS f32x4_t*)(uintptr_t)(sbase + 4 * (BM + wn * TN + 32 * j + 2 * r + 4 * (lane >> 5)));
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[i][j][r + x] = fmaf(c[r + x] * sa[i], s4[x], acc[i][j][r + x]);
        }
      } else {
        const float s = sa[i] * sb;
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(c[r], s, acc[i][j][r]);
      }
    };
    auto load_scales = [&](float (&sa)[FM], float& sb) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < FM; ++i) sa[i] = *(const LDS_AS float*)(uintptr_t)(sbase + 4 * (wm * TM + 32 * i + (lane & 31)));
      if constexpr (!ROWS)  // a wave's columns lie in one B tile
        sb = *(const LDS_AS float*)(uintptr_t)(sb0 + (t >> 3) % NSC * SB + 4 * ((t & 7) * NBT + wn * TN / 128));
    };
    float sa[FM], sb = 1.0f;
    if constexpr (WHOLE) {
      f32x16_t c[FM][FN] = {};
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        i32x8 a[FM], b[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) b[j] = b_frag(j, kk);
#pragma unroll
        for (int i = 0; i < FM; ++i) a[i] = a_frag(i, kk);
        if (kk == 1) load_scales(sa, sb);
        fence();
        __builtin_amdgcn_s_setprio(1);
        // the next sixteen of K are widened under the matrix instructions of these
        bf16x8_t w[2][FM + FN];
        auto widen = [&](int s, int n) __attribute__((always_inline)) {
          w[s & 1][n] = n < FN ? widened(b[n < FN ? n : 0], s) : widened(a[n < FN ? 0 : n - FN], s);
        };
#pragma unroll
        for (int n = 0; n < FM + FN; ++n) widen(0, n);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          fence();
#pragma unroll
          for (int m = 0; m < FM * FN; ++m) {
            const int i = m / FN, j = m % FN;
            c[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[s & 1][j], w[s & 1][FN + i], c[i][j], 0, 0, 0);
            fence();
            constexpr int EACH = (FM + FN + FM * FN - 1) / (FM * FN);
            if (s < 3)
#pragma unroll
              for (int n = m * EACH; n < m * EACH + EACH; ++n)
                if (n < FM + FN) widen(s + 1, n);
            fence();
          }
          send((NDMA + 7) / 8);
          fence();
        }
        __builtin_amdgcn_s_setprio(0);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) promote(i, j, c[i][j], sa, sb);
    } else {
      // In a fixed order (scheduling fences): a block's promotion runs under the next block's matrix
      // instructions, with two blocks and two A fragments in flight.
      auto mfma = [&](const i32x8& b, const i32x8& a, const f32x16_t& c) __attribute__((always_inline)) {
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 0, 0, 0, 127, 0, 127);
      };
      constexpr int EACH = (NDMA + 3) / 4;
      i32x8 b[2][2], a0, a1;
      b[0][0] = b_frag(0, 0);
      b[0][1] = b_frag(1, 0);
      a0 = a_frag(0, 0);
      b[1][0] = b_frag(0, 1);
      b[1][1] = b_frag(1, 1);
      a1 = a_frag(0, 1);
      load_scales(sa, sb);
      fence();
      __builtin_amdgcn_s_setprio(1);
      const f32x16_t z = {};
      f32x16_t t0 = mfma(b[0][0], a0, z), t1 = mfma(b[0][1], a0, z);
      fence();
      if (FM > 1) a0 = a_frag(1, 0);
      send(EACH);
      fence();
      t0 = mfma(b[1][0], a1, t0);
      t1 = mfma(b[1][1], a1, t1);
      fence();
      if (FM > 1) a1 = a_frag(1, 1);
      send(EACH);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        fence();
        promote(i, 0, t0, sa, sb);
        fence();
        if (i + 1 < FM) t0 = mfma(b[0][0], a0, z);
        fence();
        promote(i, 1, t1, sa, sb);
        fence();
        if (i + 1 < FM) {
          t1 = mfma(b[0][1], a0, z);
          fence();
          if (i + 2 < FM) a0 = a_frag(i + 2, 0);
          send(EACH);
          fence();
          t0 = mfma(b[1][0], a1, t0);
          t1 = mfma(b[1][1], a1, t1);
          fence();
          if (i + 2 < FM) a1 = a_frag(i + 2, 1);
          send(EACH);
        }
      }
      send(NDMA);
      __builtin_amdgcn_s_setprio(0);
    }
  };

  // ------------------------------------------------------------------ main loop
  // Stage t + S - 1 is sent in step t, and with it scales of the eight blocks behind block t + S - 2's eight:
  // what is sent in a step is complete S - 1 steps later.
  for (int id = wave; id < 8 * NG; id += NW) scales(0, id);
  if (wave == NW - 1) b_tile_scales(0);
  for (int t = 0; t < S - 1 && t < nk; ++t) {
    if (ragged && t == nk - 1) {
      dma_ragged(t);
    } else {
#pragma unroll
      for (int n = 0; n < NDMA; ++n) dma(n, t);
    }
    if (t > 0) step_scales(t - 1);
  }
  const int whole = max(nk - (S - 1) - (ragged ? 1 : 0), 0);
  for (int t = 0; t < whole; ++t) {
    vm_lgkm_wait_barrier<(S - 2) * NDMA>();  // at least S - 2 batches lie behind stage t's
    step_scales(t + S - 2);
    compute(t, std::true_type{});
  }
  for (int t = whole; t < nk; ++t) {
    if (t + S - 1 <= nk) vm_lgkm_wait_barrier<(S - 2) * NDMA>();
    else vm_lgkm_wait_barrier<0>();
    if (t + S - 1 < nk) {
      step_scales(t + S - 2);
      dma_ragged(t + S - 1);
    }
    compute(t, std::false_type{});
  }

  // ------------------------------------------------------------------ C
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int lr = wm * TM + 32 * i + (lane & 31);
    if (lr >= mrows) continue;
    const int64_t row = m0 + lr;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int col = wn * TN + 32 * j + 2 * r + 4 * (lane >> 5);
        if (col >= ncols) continue;
        float v[4] = {acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
        if (!whole_tile && cut.splits > 1)
          *(float4*)(part + ((of_k * cut.tiles + of_tile) * BM + lr) * BN + col) = make_float4(v[0], v[1], v[2], v[3]);
        else store4<WHOLE>(g, row * g.ldc + n0 + col, v);
      }
  }
}

namespace {

constexpr int kCus = 256;

// Few rows: 16 of them with any B, 48 with a B [N, K] (48x7168x2048 8.5 us, in tiles 11.7; 48x4096x8192 13.2 and
// 14.3; 40x2048x16384 15.1 and 14.4; a 64th row's operands no longer fit twice into a compute unit: 64x7168x4096
// 16.5 and 14.3).
bool is_few(const MatmulArgs& g) { return g.M <= (g.b_form == MOE_B_KN ? 16 : 48); }
// A short K with B [K, N]: 32 columns a thread block and no parts of K (1x2048x1024 3.0 us against 4.6 in 128
// columns, 1x2048x2048 5.8 and 7.3, 1x7168x2048 8.9 and 9.2); a long one takes whole lines of B
// (1x4096x7168 11.1 us against 14.2).
constexpr int kShortK = 2048;
// Columns of a thread block, and the parts of K (`per` blocks of 128 each) that make their number fill the card.
struct FewPlan {
  int64_t groups;
  int per, splits;
};
FewPlan few_plan(const MatmulArgs& g) {
  FewPlan f;
  const int KB = (int)((g.K + 127) / 128), cols = g.b_form != MOE_B_KN ? 16 : g.K <= kShortK ? 32 : 128;
  f.groups = (g.N + cols - 1) / cols;
  f.per = KB;
  if (g.K > kShortK) {
    const int64_t want = (kCus + f.groups - 1) / f.groups;
    f.per = (int)((KB + want - 1) / want);
    f.per = (f.per + 7) / 8 * 8;  // a block of K for each of the eight waves
  }
  f.splits = (KB + f.per - 1) / f.per;
  return f;
}

template <bool WHOLE>
void launch_sum(const MatmulArgs& g, const float* part, const Cut& cut, hipStream_t st) {
  const int64_t units = cut.tiles * cut.bm * cut.bn / 4;
  fp8_matmul_sum_kernel<WHOLE><<<(unsigned)((units + 255) / 256), 256, 0, st>>>(g, part, cut);
}

template <int FORM, bool WHOLE>
void launch_few_form(const MatmulArgs& g, const FewPlan& f, float* part, hipStream_t st) {
  const dim3 grid((unsigned)f.groups, (unsigned)f.splits), block(512);
  if constexpr (FORM == MOE_B_KN) {
    if (g.K <= kShortK) fp8_matmul_few_kernel<true, false, WHOLE, 1, 2, 2><<<grid, block, 0, st>>>(g, part, f.per);
    else fp8_matmul_few_kernel<true, false, WHOLE, 1, 8, 1><<<grid, block, 0, st>>>(g, part, f.per);
  } else {
    constexpr bool ROWS = FORM == MOE_B_NK_ROWS;
    if (g.M <= 16) fp8_matmul_few_kernel<false, ROWS, WHOLE, 1, 1, 4><<<grid, block, 0, st>>>(g, part, f.per);
    else if (g.M <= 32) fp8_matmul_few_kernel<false, ROWS, WHOLE, 2, 1, 1><<<grid, block, 0, st>>>(g, part, f.per);
    else fp8_matmul_few_kernel<false, ROWS, WHOLE, 3, 1, 1><<<grid, block, 0, st>>>(g, part, f.per);
  }
}

template <bool WHOLE>
void launch_few(const MatmulArgs& g, float* ws, hipStream_t st) {
  const FewPlan f = few_plan(g);
  float* part = f.splits > 1 ? ws : nullptr;
  if (g.b_form == MOE_B_KN) launch_few_form<MOE_B_KN, WHOLE>(g, f, part, st);
  else if (g.b_form == MOE_B_NK) launch_few_form<MOE_B_NK, WHOLE>(g, f, part, st);
  else launch_few_form<MOE_B_NK_ROWS, WHOLE>(g, f, part, st);
  if (part) launch_sum<WHOLE>(g, part, Cut{0, 1, f.splits, f.per, g.M, g.N, 1, 1, 1}, st);
}

// The shapes of tiles, what a step (128 of K) of a full card of them takes in ns, and where two fit a compute unit,
// also of one each (measured: 4096x4096x4096 and 7168x4096x21808 in every shape, 2048x2048x7168 for the last).
struct Shape {
  int bm, bn, per_cu, step, step_alone;
};
constexpr Shape kShapes[2][4] = {  // bf16 C, fp32 C
    {{256, 256, 1, 2080, 2080}, {256, 128, 1, 1330, 1330}, {128, 128, 2, 1320, 930}, {64, 128, 2, 900, 600}},
    {{256, 128, 1, 2250, 2250}, {128, 128, 2, 2500, 1750}, {64, 128, 2, 1300, 900}, {0, 0, 0, 0, 0}}};

// The shape, and into how many parts of K the tiles behind the last full card are cut, by the time that the steps
// take, 3 us for each round of tiles, and 3 us and both ways of the parts' bytes at 5 TB/s for the sums:
// 21804x4096x7168, 1376 tiles of 256 x 256: 96 cut in two, 5.5 rounds instead of 6 (650 -> 640 us); 7168x4096x21808 in
// fp32, 896 of 256 x 128: 128 cut in two, 3.5 instead of 4 (1434 -> 1351 us).  Shapes against each other, bf16, in us:
// 1023x7168x4096 256x256 55, 256x128 43, 128x128 45, 64x128 54; 4096x4096x4096 74, 91, 89, 112; 300x8192x8192 53, 59, 56, 47.
Cut tile_plan(const MatmulArgs& g) {
  const int KB = (int)((g.K + 127) / 128);
  Cut best{};
  double least = 0.0;
  for (const Shape& sh : kShapes[g.c_f32]) {
    if (sh.bm == 0) continue;
    Cut c{};
    c.bm = sh.bm, c.bn = sh.bn, c.gm = 8;
    c.nM = (int)((g.M + sh.bm - 1) / sh.bm), c.nN = (int)((g.N + sh.bn - 1) / sh.bn);
    const int64_t all = (int64_t)c.nM * c.nN, slots = kCus * sh.per_cu, rem = all % slots;
    const double full = (double)(all / slots) * ((double)KB * sh.step + 3e3);
    for (int want = 1; want == 1 || (want * rem <= slots && KB >= 4 * want); ++want) {
      c.per = (KB + want - 1) / want;
      c.splits = (KB + c.per - 1) / c.per;
      c.tiles = c.splits > 1 ? rem : 0;
      c.first = all - c.tiles;
      double t = full;
      if (rem > 0) {  // between one and two a compute unit: between both times
        const double two = rem * c.splits > kCus ? (double)(rem * c.splits - kCus) / kCus : 0.0;
        t += c.per * (sh.step_alone + two * (sh.step - sh.step_alone)) + 3e3;
      }
      if (c.tiles > 0) t += 3e3 + (double)(c.tiles * c.splits) * sh.bm * sh.bn * 8 / 5e3;
      if (least == 0.0 || t < least) least = t, best = c;
      if (rem == 0) break;
    }
  }
  return best;
}

template <int FORM, bool WHOLE>
void launch_tiles_form(const MatmulArgs& g, const Cut& c, float* part, hipStream_t st) {
  const unsigned grid = (unsigned)(c.first + c.tiles * c.splits);
  if (c.bm == 256 && c.bn == 128) fp8_matmul_tile_kernel<FORM, WHOLE, 256, 128, 4, 2, 2><<<grid, 512, 0, st>>>(g, part, c);
  else if (c.bm == 256) {
    if constexpr (!WHOLE) fp8_matmul_tile_kernel<FORM, false, 256, 256, 2, 4, 2><<<grid, 512, 0, st>>>(g, part, c);
  }
  else if (c.bm == 128) fp8_matmul_tile_kernel<FORM, WHOLE, 128, 128, 2, 2, 2><<<grid, 256, 0, st>>>(g, part, c);
  else fp8_matmul_tile_kernel<FORM, WHOLE, 64, 128, 2, 2, FORM == MOE_B_NK_ROWS ? 2 : 3><<<grid, 256, 0, st>>>(g, part, c);
}

template <bool WHOLE>
void launch_tiles(const MatmulArgs& g, float* ws, hipStream_t st) {
  const Cut c = tile_plan(g);
  if (g.b_form == MOE_B_KN) launch_tiles_form<MOE_B_KN, WHOLE>(g, c, ws, st);
  else if (g.b_form == MOE_B_NK) launch_tiles_form<MOE_B_NK, WHOLE>(g, c, ws, st);
  else launch_tiles_form<MOE_B_NK_ROWS, WHOLE>(g, c, ws, st);
  if (c.tiles > 0) launch_sum<WHOLE>(g, ws, c, st);
}

}  // namespace

size_t fp8_matmul_ws_bytes(const MatmulArgs& g) {
  if (g.M == 0) return 0;
  if (is_few(g)) {
    const int splits = few_plan(g).splits;
    return splits > 1 ? (size_t)splits * g.M * g.N * sizeof(float) : 0;
  }
  const Cut c = tile_plan(g);
  return (size_t)(c.tiles * c.splits * c.bm * c.bn) * sizeof(float);
}

hipError_t launch_fp8_matmul(const MatmulArgs& g, void* ws, hipStream_t st) {
  if (is_few(g)) {
    if (g.c_f32) launch_few<true>(g, (float*)ws, st);
    else launch_few<false>(g, (float*)ws, st);
  } else {
    if (g.c_f32) launch_tiles<true>(g, (float*)ws, st);
    else launch_tiles<false>(g, (float*)ws, st);
  }
  return hipGetLastError();
}

}  // namespace moe
