// Dense products of blockwise e4m3 operands on gfx950's fp8 MFMA (v_mfma_scale_f32_32x32x64_f8f6f4 with
// unit block exponents): C = A . B (+ C_in) with one scale per row and 128 values of K for A, and for B
// one per 128 x 128 block or one per row and 128 values.  Blockwise FP8 is one of the data types of the
// fused MoE backward on the Prime Mega MoE page ("Prime Mega MoE: tanításra is jó a DeepSeek MoE
// kernele", section "Mit csinált a Prime Intellect?").
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
// Up to 16 rows: the product is a reading of B.  A wave takes whole blocks of K (128 deep) of a few
// columns, its own ones, so that no wave waits for another until the end: B by DMA into LDS of the
// wave's own, whole cache lines a row (a load that takes 64 bytes of 16 rows ran at half the rate), A's
// rows into registers from L2.  The waves' sums meet in LDS in a fixed order; where the columns alone
// give too few thread blocks, K is cut once more over `splits` of them, whose fp32 sums
// fp8_matmul_sum_kernel adds in order.
//
// B [N, K]: 16 NF columns a thread block, whose eight waves take the blocks of K in turn, U at a time.
// B [K, N]: 128 columns, one cache line, and four waves; the LDS transpose read makes the operands.
constexpr int kFewRows = 16;

template <bool KN, bool ROWS, bool WHOLE, int MF, int NF, int U, int CW>
__global__ __launch_bounds__(512) void fp8_matmul_few_kernel(const MatmulArgs g, float* __restrict__ part,
                                                                        int per) {
  constexpr int KW = 8 / CW;           // waves that share K; CW of them stand side by side
  constexpr int BLK = 2048 * NF;       // bytes of a block of K
  static_assert(!KN || !ROWS, "");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[8 * U * BLK];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave / CW;
  const int64_t nblk = (int64_t)xcd_remap(blockIdx.x, gridDim.x) * (16 * NF * CW), n0 = nblk + 16 * NF * (wave % CW);
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
  };
  struct Row {
    i32x8 a[MF];
    float sa[MF], sb[ROWS ? 4 * NF : KN ? 1 : NF];
  };
  // the 32 bytes of K that lane l has of its row: 16-byte pieces q and q + 4 of the block
  auto load = [&](Row& c, int kb) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)kb * 128 + 16 * q;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      u32x4 lo = {}, hi = {};
      if (k0 < g.K) lo = *(const u32x4*)(a_row[i] + k0);
      if (k0 + 64 < g.K) hi = *(const u32x4*)(a_row[i] + k0 + 64);
      c.a[i] = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
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
        const u32x4 lo = *(const LDS_AS u32x4*)(uintptr_t)(base + km_off<64>(16 * j + l16, q));
        const u32x4 hi = *(const LDS_AS u32x4*)(uintptr_t)(base + km_off<64>(16 * j + l16, q + 4));
        b = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
      }
      // the last block: a NaN code would outlive A's zero
#pragma unroll
      for (int w = 0; w < 8; ++w)
        if (left <= 64 * (w >> 2)) b[w] = 0;
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const f32x4_t t = multiply16<WHOLE>(b, c.a[i]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(t[r], c.sa[i] * c.sb[ROWS ? 4 * j + r : KN ? 0 : j], acc[i][j][r]);
      }
    }
  };
  for (int kb = kb0 + kw; kb < kb1; kb += KW * U) {
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
  constexpr int UNITS = CW * NF * 64;
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
      const int64_t m = 16 * i + (u & 15), n = nblk + 16 * (u >> 6) + 4 * ((u & 63) >> 4);
      if (m >= g.M || n >= g.N) continue;
      if (part) *(float4*)(part + ((int64_t)blockIdx.y * g.M + m) * g.N + n) = make_float4(v[0], v[1], v[2], v[3]);
      else store4<WHOLE>(g, m * g.ldc + n, v);
    }
  }
}

// The sums of the parts of K, in order; four values a thread.
template <bool F32>
__global__ __launch_bounds__(256) void fp8_matmul_sum_kernel(const MatmulArgs g, const float* __restrict__ part,
                                                             int splits) {
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u * 4 >= g.M * g.N) return;
  const int64_t m = u * 4 / g.N, n = u * 4 - m * g.N;
  float v[4] = {};
  for (int s0 = 0; s0 < splits; s0 += 8) {  // eight loads in flight
    float4 a[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) a[s] = *(const float4*)(part + min(s0 + s, splits - 1) * g.M * g.N + u * 4);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s0 + s < splits) v[0] += a[s].x, v[1] += a[s].y, v[2] += a[s].z, v[3] += a[s].w;
  }
  store4<F32>(g, m * g.ldc + n, v);
}

// -------------------------------------------------------------------------------------- tiles
// What a tile kernel reads in the place of codes past K.
__device__ const uint4 g_zero = {0, 0, 0, 0};

// BM x BN tiles, WM x WN waves, a block of K (128 deep) a step through S LDS stages.  Operands and scales
// reach LDS by DMA; the number of DMAs a wave issues in a step is fixed, so that the wait for a stage
// counts those of the stages behind it.
//
// Scales.  A row's scales lie along K, so the 4 bytes a step needs of a row come with a cache line of
// their own.  Scales are therefore fetched for eight blocks of K at a time, during the eight steps before
// they are used: in step t each wave brings, for one block of K of the next eight, the scales of 32 rows; the
// waves of a step share the rows, and with them the lines.  The scale of a B tile rides in the lanes behind.
//
// Each 32 x 32 block of C is held transposed (B is the MFMA's first operand): lane l has row l % 32 and 16
// columns, so one A scale serves its 16 values.
template <int FORM, bool WHOLE, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN, 1) void fp8_matmul_tile_kernel(const MatmulArgs g, float* __restrict__ part, int per,
                                                                          int gm) {
  constexpr bool KN = FORM == MOE_B_KN, ROWS = FORM == MOE_B_NK_ROWS;
  constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32, BK = 128;
  constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
  constexpr int QA = A_BYTES / 1024 / NW, QB = B_BYTES / 1024 / NW;
  constexpr int NG = (BM + (ROWS ? BN : 0)) / 32;      // groups of 32 rows with scales
  constexpr int UPW = (NG + NW - 1) / NW;              // scale DMAs a wave and step
  constexpr int SLOT = ROWS ? 128 : 144;               // bytes of a group's scales: 32 rows, up to 4 B tiles
  constexpr int SC = 8 * NG * SLOT, NSC = S > 2 ? 3 : 2;  // of eight blocks of K; how many of those there are
  constexpr int NDMA = QA + QB + UPW;
  static_assert(QA * 1024 * NW == A_BYTES && QB * 1024 * NW == B_BYTES, "DMA split");
  static_assert(!KN || BN == 128 || BN == 256, "[K, N] layouts");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE + NSC * SC];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr_of(smem)), sc0 = lds0 + S * STAGE;
  const int nM = (int)((g.M + BM - 1) / BM), nN = (int)((g.N + BN - 1) / BN);
  const int2 tile = grouped_tile(xcd_remap(blockIdx.x, gridDim.x), nM, nN, gm);
  const int64_t m0 = (int64_t)tile.x * BM, n0 = (int64_t)tile.y * BN;
  const int KB = (int)((g.K + 127) / 128);
  const int64_t NB = (g.N + 127) / 128;
  const int kb0 = blockIdx.y * per, nk = min(KB - kb0, per);

  // ------------------------------------------------------------------ DMA sources
  const uint8_t* a_src[QA];
  const uint8_t* b_src[QB];
  int a_k[QA], b_k[QB];  // first code of K within the block
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int row = 8 * (wave * QA + q) + lane / 8, c = (lane % 8) ^ ((row >> 1) & 7);
    a_k[q] = 16 * c;
    a_src[q] = g.A + min(m0 + row, g.M - 1) * g.lda + (int64_t)kb0 * BK + a_k[q];
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    if constexpr (KN) {
      constexpr int RPD = 1024 / BN;  // K rows a DMA
      const int kr = RPD * (wave * QB + q) + lane / (BN / 16), cl = lane % (BN / 16);
      const int c = BN == 256 ? cl ^ (2 * (kr & 7)) : cl ^ (2 * ((kr >> 1) & 3));
      b_k[q] = kr;
      b_src[q] = g.B + ((int64_t)kb0 * BK + kr) * g.ldb + min(n0 + 16 * c, g.N - 16);
    } else {
      const int row = 8 * (wave * QB + q) + lane / 8, c = (lane % 8) ^ ((row >> 1) & 7);
      b_k[q] = 16 * c;
      b_src[q] = g.B + min(n0 + row, g.N - 1) * g.ldb + (int64_t)kb0 * BK + b_k[q];
    }
  }
  const bool ragged = g.K % BK != 0;
  auto issue = [&](int t, int st) __attribute__((always_inline)) {
    const uint32_t abase = lds0 + st * STAGE, bbase = abase + A_BYTES;
    const int64_t k0 = (int64_t)t * BK;
    if (ragged && kb0 + t == KB - 1) {
      const int left = (int)(g.K - (int64_t)(KB - 1) * BK);
#pragma unroll
      for (int q = 0; q < QA; ++q)
        dma16(a_k[q] < left ? (const void*)(a_src[q] + k0) : (const void*)&g_zero, abase + (wave * QA + q) * 1024);
#pragma unroll
      for (int q = 0; q < QB; ++q)
        dma16(b_k[q] < left ? (const void*)(b_src[q] + (KN ? k0 * g.ldb : k0)) : (const void*)&g_zero,
              bbase + (wave * QB + q) * 1024);
    } else {
#pragma unroll
      for (int q = 0; q < QA; ++q) dma16(a_src[q] + k0, abase + (wave * QA + q) * 1024);
#pragma unroll
      for (int q = 0; q < QB; ++q) dma16(b_src[q] + (KN ? k0 * g.ldb : k0), bbase + (wave * QB + q) * 1024);
    }
  };
  // scales of group grp (A's rows, then B's) for block k of the chunk at block k8 of the thread block's own
  auto scales = [&](int k8, int k, int grp) __attribute__((always_inline)) {
    const int kb = min(kb0 + k8 + k, KB - 1);
    const float* src;
    if (lane < 32 || ROWS) {
      const bool of_b = ROWS && grp >= BM / 32;
      const int64_t row = of_b ? min(n0 + 32 * (grp - BM / 32) + (lane & 31), g.N - 1) : min(m0 + 32 * grp + (lane & 31), g.M - 1);
      src = (of_b ? g.B_scale : g.A_scale) + row * KB + kb;
    } else {
      const int64_t nb = min(n0 / 128 + (lane - 32), NB - 1);
      src = g.B_scale + (KN ? kb * NB + nb : nb * KB + kb);
    }
    if (lane < (ROWS ? 32 : 32 + BN / 128)) dma4(src, sc0 + (k8 >> 3) % NSC * SC + (k * NG + grp) * SLOT);
  };

  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x16_t{};

  auto compute = [&](int t, int st) __attribute__((always_inline)) {
    const uint32_t abase = lds0 + st * STAGE, bbase = abase + A_BYTES;
    const uint32_t sbase = sc0 + (t >> 3) % NSC * SC + (t & 7) * NG * SLOT;
    auto b_frag = [&](int j, int kk) __attribute__((always_inline)) -> i32x8 {
      const int col = wn * TN + 32 * j;
      if constexpr (KN && BN == 256) return read_kn8(bbase, col, kk, lane);
      else if constexpr (KN) return read_kn8n(bbase, col, kk, lane);
      else return read_km8(bbase, col + (lane & 31), kk, lane);
    };
    i32x8 b[2][FN];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int j = 0; j < FN; ++j) b[kk][j] = b_frag(j, kk);
    float sa[FM], sb[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = *(const LDS_AS float*)(uintptr_t)(sbase + (wm * FM + i) * SLOT + 4 * (lane & 31));
#pragma unroll
    for (int j = 0; j < FN; ++j)
      if constexpr (!ROWS) sb[j] = *(const LDS_AS float*)(uintptr_t)(sbase + 128 + 4 * ((wn * TN + 32 * j) / 128));
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = wm * TM + 32 * i + (lane & 31);
      const i32x8 a0 = read_km8(abase, row, 0, lane), a1 = read_km8(abase, row, 1, lane);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        f32x16_t c = multiply<WHOLE>(b[0][j], a0, f32x16_t{});
        c = multiply<WHOLE>(b[1][j], a1, c);
        if constexpr (ROWS) {
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const f32x4_t s4 = *(const LDS_AS f32x4_t*)(uintptr_t)(sbase + (BM / 32 + (wn * TN) / 32 + j) * SLOT +
                                                                  4 * (8 * (r >> 2) + 4 * (lane >> 5)));
            acc[i][j][r] = fmaf(c[r] * sa[i], s4[0], acc[i][j][r]);
            acc[i][j][r + 1] = fmaf(c[r + 1] * sa[i], s4[1], acc[i][j][r + 1]);
            acc[i][j][r + 2] = fmaf(c[r + 2] * sa[i], s4[2], acc[i][j][r + 2]);
            acc[i][j][r + 3] = fmaf(c[r + 3] * sa[i], s4[3], acc[i][j][r + 3]);
          }
        } else {
          const float s = sa[i] * sb[j];
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(c[r], s, acc[i][j][r]);
        }
      }
    }
  };

  // ------------------------------------------------------------------ main loop
  // A batch: a stage's operands, and the wave's share of the scales of the eight blocks behind block t's
  // eight, where all (group, block) pairs are numbered with the blocks first.
  auto batch = [&](int stage, int t) __attribute__((always_inline)) {
    issue(stage, stage % S);
#pragma unroll
    for (int u = 0; u < UPW; ++u) {
      const int id = min(((t & 7) * UPW + u) * NW + wave, 8 * NG - 1);
      scales((t & ~7) + 8, id & 7, id >> 3);
    }
  };
  for (int id = wave; id < 8 * NG; id += NW) scales(0, id & 7, id >> 3);
  for (int t = 0; t < S - 1 && t < nk; ++t) batch(t, max(t - 1, 0));
  for (int t = 0; t < nk; ++t) {
    if (t + S - 1 <= nk) vm_lgkm_wait_barrier<(S - 2) * NDMA>();  // S - 2 batches lie behind stage t's
    else vm_lgkm_wait_barrier<0>();
    // the batch of step t is complete in step t + S - 1: the scales of a chunk's first block go out S - 2 steps ahead
    if (t + S - 1 < nk) batch(t + S - 1, t + S - 2);
    compute(t, t % S);
  }
  vm_wait<0>();  // no DMA outlives the thread block

  // ------------------------------------------------------------------ C
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t row = m0 + wm * TM + 32 * i + (lane & 31);
    if (row >= g.M) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int64_t col = n0 + wn * TN + 32 * j + 8 * (r >> 2) + 4 * (lane >> 5);
        if (col >= g.N) continue;
        float v[4] = {acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
        if (part) *(float4*)(part + ((int64_t)blockIdx.y * g.M + row) * g.N + col) = make_float4(v[0], v[1], v[2], v[3]);
        else store4<WHOLE>(g, row * g.ldc + col, v);
      }
  }
}

namespace {

// Few rows: columns of a thread block, and the parts of K (`per` blocks of 128 each) that make their
// number fill the card.
struct FewPlan {
  int nf;
  int64_t groups;
  int per, splits;
};
#ifndef WANT
#define WANT 256
#define NFS 1
#define CWK 2
#endif
FewPlan few_plan(const MatmulArgs& g) {
  FewPlan f;
  const int KB = (int)((g.K + 127) / 128);
  const bool wide = g.b_form == MOE_B_KN;
  f.nf = wide ? 8 * CWK : g.M <= 16 ? NFS : 2;
  f.groups = (g.N + 16 * f.nf - 1) / (16 * f.nf);
  const int waves = wide ? 8 / CWK : 8;
  const int64_t want = (WANT + f.groups - 1) / f.groups;
  f.per = (int)((KB + want - 1) / want);
  f.per = (f.per + waves - 1) / waves * waves;
  f.splits = (KB + f.per - 1) / f.per;
  return f;
}

template <bool KN, bool ROWS, bool WHOLE>
void launch_few_form(const MatmulArgs& g, const FewPlan& f, float* part, hipStream_t st) {
  const dim3 grid((unsigned)f.groups, (unsigned)f.splits), block(512);
  if constexpr (KN) fp8_matmul_few_kernel<KN, ROWS, WHOLE, 1, 8, 1, 2><<<grid, block, 0, st>>>(g, part, f.per);
  else fp8_matmul_few_kernel<KN, ROWS, WHOLE, 1, 1, 4, 1><<<grid, block, 0, st>>>(g, part, f.per);
}

template <bool WHOLE>
void launch_few(const MatmulArgs& g, float* ws, hipStream_t st) {
  const FewPlan f = few_plan(g);
  float* part = f.splits > 1 ? ws : nullptr;
  if (g.b_form == MOE_B_KN) launch_few_form<true, false, WHOLE>(g, f, part, st);
  else if (g.b_form == MOE_B_NK) launch_few_form<false, false, WHOLE>(g, f, part, st);
  else launch_few_form<false, true, WHOLE>(g, f, part, st);
  if (part)
    fp8_matmul_sum_kernel<WHOLE><<<(unsigned)((g.M * g.N / 4 + 255) / 256), 256, 0, st>>>(g, part, f.splits);
}

// Tiles: rows, columns, parts of K.
struct TilePlan {
  int bm, bn;
  int per, splits;
};
TilePlan tile_plan(const MatmulArgs& g) {
  TilePlan f;
  const int KB = (int)((g.K + 127) / 128);
  auto tiles = [&](int bm, int bn) { return (g.M + bm - 1) / bm * ((g.N + bn - 1) / bn); };
  if (tiles(256, 256) >= 192) {
    f.bm = f.bn = 256;
  } else {
    f.bm = g.M <= 64 ? 64 : 128;
    f.bn = 128;
  }
  f.per = KB;
  if (f.bm < 256) {
    const int64_t want = (256 + tiles(f.bm, f.bn) - 1) / tiles(f.bm, f.bn);
    f.per = (int)((KB + want - 1) / want);
    if (f.per < 4) f.per = KB < 4 ? KB : 4;
  }
  f.splits = (KB + f.per - 1) / f.per;
  return f;
}

template <int FORM, bool WHOLE>
void launch_tiles_form(const MatmulArgs& g, const TilePlan& f, float* part, hipStream_t st) {
  const dim3 grid((unsigned)((g.M + f.bm - 1) / f.bm * ((g.N + f.bn - 1) / f.bn)), (unsigned)f.splits);
  if (f.bm == 256) fp8_matmul_tile_kernel<FORM, WHOLE, 256, 256, 2, 4, 2><<<grid, 512, 0, st>>>(g, part, f.per, 8);
  else if (f.bm == 128) fp8_matmul_tile_kernel<FORM, WHOLE, 128, 128, 2, 2, 3><<<grid, 256, 0, st>>>(g, part, f.per, 8);
  else fp8_matmul_tile_kernel<FORM, WHOLE, 64, 128, 1, 4, 4><<<grid, 256, 0, st>>>(g, part, f.per, 8);
}

template <bool WHOLE>
void launch_tiles(const MatmulArgs& g, float* ws, hipStream_t st) {
  const TilePlan f = tile_plan(g);
  float* part = f.splits > 1 ? ws : nullptr;
  if (g.b_form == MOE_B_KN) launch_tiles_form<MOE_B_KN, WHOLE>(g, f, part, st);
  else if (g.b_form == MOE_B_NK) launch_tiles_form<MOE_B_NK, WHOLE>(g, f, part, st);
  else launch_tiles_form<MOE_B_NK_ROWS, WHOLE>(g, f, part, st);
  if (part)
    fp8_matmul_sum_kernel<WHOLE><<<(unsigned)((g.M * g.N / 4 + 255) / 256), 256, 0, st>>>(g, part, f.splits);
}

}  // namespace

size_t fp8_matmul_ws_bytes(const MatmulArgs& g) {
  if (g.M == 0) return 0;
  const int splits = g.M <= kFewRows ? few_plan(g).splits : tile_plan(g).splits;
  return splits > 1 ? (size_t)splits * g.M * g.N * sizeof(float) : 0;
}

hipError_t launch_fp8_matmul(const MatmulArgs& g, void* ws, hipStream_t st) {
  if (g.M <= kFewRows) {
    if (g.c_f32) launch_few<true>(g, (float*)ws, st);
    else launch_few<false>(g, (float*)ws, st);
  } else {
    if (g.c_f32) launch_tiles<true>(g, (float*)ws, st);
    else launch_tiles<false>(g, (float*)ws, st);
  }
  return hipGetLastError();
}

}  // namespace moe
