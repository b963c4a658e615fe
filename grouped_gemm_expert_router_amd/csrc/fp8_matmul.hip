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
// Up to 64 rows: the product is a reading of B.  Every wave takes whole blocks of K of a few columns
// straight into registers (no LDS, nothing to wait for but the loads), all 64 rows of A beside them
// from L2, and the waves' sums meet in LDS in a fixed order; where columns alone give too few thread
// blocks, K is cut again over `splits` of them, whose fp32 sums few_sum_kernel adds in order.
//
// B [N, K]: a block of eight waves has 16 NF columns; wave w takes the blocks of K w, w + 8, ...  Lane l
// holds row l % 16 and, of a block's eight 16-byte pieces, l / 16 and l / 16 + 4: a load reads 64
// neighbouring bytes of 16 rows.
// B [K, N]: a block has 128 columns, one cache line; of its eight waves, two halves of 64 columns times
// four blocks of K.  Lane l loads the four codes of columns 4 (l % 16) of 32 rows of K, 64 bytes of a row
// with 16 lanes, and 4 x 4 byte transposes make of them the operands of four products, whose columns
// are 4 (l % 16) + i.
constexpr int kFewRows = 64;

template <bool KN, bool ROWS, bool WHOLE, int MF, int NF>
__global__ __launch_bounds__(512) void fp8_matmul_few_kernel(const MatmulArgs g, float* __restrict__ part, int per) {
  constexpr int KW = KN ? 4 : 8;              // waves that share K
  constexpr int CW = KN ? 64 : 16 * NF;       // columns of a wave
  constexpr int U = KN ? 1 : MF + NF <= 2 ? 4 : MF + NF <= 4 ? 2 : 1;  // blocks of K loaded ahead
  static_assert(!KN || (NF == 4 && !ROWS), "64 columns of a [K, N] operand");
  __shared__ float4 red[8 * MF * NF * 64];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = KN ? wave >> 1 : wave;
  const int64_t n0 = (int64_t)blockIdx.x * (KN ? 128 : CW) + (KN ? (wave & 1) * 64 : 0);
  const int KB = (int)((g.K + 127) / 128);
  const int64_t NB = (g.N + 127) / 128;
  const int kb0 = blockIdx.y * per, kb1 = min(KB, kb0 + per);
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

  struct Block {
    i32x8 a[MF], b[NF];  // KN: b[j / 8][j % 8] is the word of K row j
    float sa[MF], sb[ROWS ? 4 * NF : NF];
  };
  // 32 bytes of a row: pieces q and q + 4 of the block at k0
  auto pieces = [&](const uint8_t* row, int64_t k0) __attribute__((always_inline)) {
    u32x4 v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = k0 + 64 * h + 16 * q;
      v[h] = u32x4{};
      if (k < g.K) v[h] = *(const u32x4*)(row + k);
    }
    return i32x8{(int)v[0].x, (int)v[0].y, (int)v[0].z, (int)v[0].w, (int)v[1].x, (int)v[1].y, (int)v[1].z, (int)v[1].w};
  };
  auto load = [&](Block& c, int kb) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)kb * 128;
    if constexpr (KN) {
      const int64_t col = min(n0 + 4 * l16, g.N - 4);  // columns past the last feed unstored values
      const uint8_t* p = g.B + (k0 + 16 * q) * g.ldb + col;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = k0 + 64 * h + 16 * q < g.K;  // K is a multiple of 16
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int w = 16 * h + j;
          c.b[w / 8][w % 8] = 0;
          if (in) c.b[w / 8][w % 8] = *(const int*)(p + (64 * h + j) * g.ldb);
        }
      }
      c.sb[0] = g.B_scale[kb * NB + blockIdx.x];
    } else {
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const int64_t n = min(n0 + 16 * j, g.N - 16);
        c.b[j] = pieces(g.B + (n + l16) * g.ldb, k0);
        if constexpr (ROWS) {
#pragma unroll
          for (int r = 0; r < 4; ++r) c.sb[4 * j + r] = g.B_scale[(n + 4 * q + r) * KB + kb];
        } else {
          c.sb[j] = g.B_scale[n / 128 * KB + kb];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      c.a[i] = pieces(a_row[i], k0);
      c.sa[i] = a_scale[i][kb];
    }
  };
  auto add = [&](const Block& c) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      i32x8 b;
      if constexpr (KN) {
        // byte j of each word: K rows 4w .. 4w+3 of column 4 (l % 16) + j
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const uint32_t w0 = c.b[w / 2][4 * (w & 1)], w1 = c.b[w / 2][4 * (w & 1) + 1], w2 = c.b[w / 2][4 * (w & 1) + 2],
                         w3 = c.b[w / 2][4 * (w & 1) + 3];
          const uint32_t sel = j == 0 ? 0x0c0c0400u : j == 1 ? 0x0c0c0501u : j == 2 ? 0x0c0c0602u : 0x0c0c0703u;
          const uint32_t lo = __builtin_amdgcn_perm(w1, w0, sel), hi = __builtin_amdgcn_perm(w3, w2, sel);
          b[w] = (int)__builtin_amdgcn_perm(hi, lo, 0x05040100u);
        }
      } else {
        b = c.b[j];
      }
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const f32x4_t t = multiply16<WHOLE>(b, c.a[i]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(t[r], c.sa[i] * c.sb[ROWS ? 4 * j + r : KN ? 0 : j], acc[i][j][r]);
      }
    }
  };
  for (int kb = kb0 + kw; kb < kb1; kb += KW * U) {
    Block c[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kb + KW * u < kb1) load(c[u], kb + KW * u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kb + KW * u < kb1) add(c[u]);
  }
  // four neighbouring columns of a row a lane: [N, K] 4q + 0..3 of fragment j; [K, N] 16q + 4j + 0..3
  const int half = KN ? wave & 1 : 0;
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      float4 v;
      if constexpr (KN) v = make_float4(acc[i][0][j], acc[i][1][j], acc[i][2][j], acc[i][3][j]);
      else v = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
      red[((kw * (8 / KW) + half) * MF * NF + i * NF + j) * 64 + lane] = v;
    }
  __syncthreads();
  constexpr int UNITS = (8 / KW) * MF * NF * 64;
  for (int u = threadIdx.x; u < UNITS; u += 512) {
    float v[4] = {};
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const float4 a = red[k * UNITS + u];
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    }
    const int ul = u & 63, j = u / 64 % NF, i = u / 64 / NF % MF, h = u / 64 / NF / MF;
    const int64_t m = 16 * i + (ul & 15);
    const int64_t n = (int64_t)blockIdx.x * (KN ? 128 : CW) +
                      (KN ? 64 * h + 16 * (ul >> 4) + 4 * j : 16 * j + 4 * (ul >> 4));
    if (m >= g.M || n >= g.N) continue;
    if (part) *(float4*)(part + ((int64_t)blockIdx.y * g.M + m) * g.N + n) = make_float4(v[0], v[1], v[2], v[3]);
    else store4<WHOLE>(g, m * g.ldc + n, v);
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
  for (int s = 0; s < splits; ++s) {
    const float4 a = *(const float4*)(part + s * g.M * g.N + u * 4);
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
  }
  store4<F32>(g, m * g.ldc + n, v);
}

// 128 x 128 tiles, four waves of 64 x 64, one block of K a step through one LDS stage.  Each 32 x 32
// block of C is held transposed (B is the MFMA's first operand): lane l has row l % 32 and 16 columns.
template <int FORM, bool WHOLE>
__global__ __launch_bounds__(256) void fp8_matmul_tile_kernel(const MatmulArgs g) {
  constexpr int BM = 128, BN = 128, BK = 128;
  constexpr bool KN = FORM == MOE_B_KN, ROWS = FORM == MOE_B_NK_ROWS;
  __shared__ __attribute__((aligned(1024))) uint8_t sh_a[BM * BK];
  __shared__ __attribute__((aligned(1024))) uint8_t sh_b[BN * BK];
  __shared__ __attribute__((aligned(16))) float sh_sa[BM], sh_sb[BN];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  const int64_t nN = (g.N + BN - 1) / BN;
  const int64_t m0 = blockIdx.x / nN * BM, n0 = blockIdx.x % nN * BN;
  const int64_t KB = (g.K + 127) / 128, NB = (g.N + 127) / 128;
  const uint32_t abase = lds_addr_of(sh_a), bbase = lds_addr_of(sh_b);
  f32x16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  for (int64_t kb = 0; kb < KB; ++kb) {
    const int64_t k0 = kb * BK;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = tid + 256 * i, row = q / 8, c = q % 8;
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (m0 + row < g.M && k0 + 16 * c < g.K) a = *(const uint4*)(g.A + (m0 + row) * g.lda + k0 + 16 * c);
      if constexpr (KN) {
        if (k0 + row < g.K && n0 + 16 * c < g.N) b = *(const uint4*)(g.B + (k0 + row) * g.ldb + n0 + 16 * c);
        *(LDS_AS u32x4*)(uintptr_t)(bbase + kn8n_off(row, 16 * c)) = u32x4{b.x, b.y, b.z, b.w};
      } else {
        if (n0 + row < g.N && k0 + 16 * c < g.K) b = *(const uint4*)(g.B + (n0 + row) * g.ldb + k0 + 16 * c);
        *(LDS_AS u32x4*)(uintptr_t)(bbase + km_off<64>(row, c)) = u32x4{b.x, b.y, b.z, b.w};
      }
      *(LDS_AS u32x4*)(uintptr_t)(abase + km_off<64>(row, c)) = u32x4{a.x, a.y, a.z, a.w};
    }
    if (tid < BM) sh_sa[tid] = m0 + tid < g.M ? g.A_scale[(m0 + tid) * KB + kb] : 0.0f;
    if (ROWS && tid >= BM) sh_sb[tid - BM] = n0 + tid - BM < g.N ? g.B_scale[(n0 + tid - BM) * KB + kb] : 0.0f;
    const float sb = ROWS ? 1.0f : g.B_scale[KN ? kb * NB + n0 / 128 : n0 / 128 * KB + kb];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f32x16_t t = {};
        const int col = 64 * wn + 32 * j;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const i32x8 a = read_km8(abase, 64 * wm + 32 * i + (lane & 31), kk, lane);
          i32x8 b;
          if constexpr (KN) b = read_kn8n(bbase, col, kk, lane);
          else b = read_km8(bbase, col + (lane & 31), kk, lane);
          t = multiply<WHOLE>(b, a, t);
        }
        const float sa = sh_sa[64 * wm + 32 * i + (lane & 31)] * sb;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float s = ROWS ? sa * sh_sb[col + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)] : sa;
          acc[i][j][r] = fmaf(t[r], s, acc[i][j][r]);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = m0 + 64 * wm + 32 * i + (lane & 31);
    if (row >= g.M) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int64_t col = n0 + 64 * wn + 32 * j + 8 * (r >> 2) + 4 * (lane >> 5);
        if (col >= g.N) continue;
        float v[4] = {acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
        store4<WHOLE>(g, row * g.ldc + col, v);
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
FewPlan few_plan(const MatmulArgs& g) {
  FewPlan f;
  const int KB = (int)((g.K + 127) / 128);
  const bool kn = g.b_form == MOE_B_KN;
  f.nf = kn ? 4 : g.M <= 16 ? 1 : 2;
  f.groups = kn ? (g.N + 127) / 128 : (g.N + 16 * f.nf - 1) / (16 * f.nf);
  const int waves = kn ? 4 : 8;  // that share K in a thread block
  const int64_t want = (256 + f.groups - 1) / f.groups;  // thread blocks a compute unit: one
  f.per = (int)((KB + want - 1) / want);
  f.per = (f.per + waves - 1) / waves * waves;
  f.splits = (KB + f.per - 1) / f.per;
  return f;
}

template <bool KN, bool ROWS, bool WHOLE, int NF>
void launch_few_mf(const MatmulArgs& g, const FewPlan& f, float* part, hipStream_t st) {
  const dim3 grid((unsigned)f.groups, (unsigned)f.splits);
  if (g.M <= 16) fp8_matmul_few_kernel<KN, ROWS, WHOLE, 1, NF><<<grid, 512, 0, st>>>(g, part, f.per);
  else if (g.M <= 32) fp8_matmul_few_kernel<KN, ROWS, WHOLE, 2, NF><<<grid, 512, 0, st>>>(g, part, f.per);
  else if (g.M <= 48) fp8_matmul_few_kernel<KN, ROWS, WHOLE, 3, NF><<<grid, 512, 0, st>>>(g, part, f.per);
  else fp8_matmul_few_kernel<KN, ROWS, WHOLE, 4, NF><<<grid, 512, 0, st>>>(g, part, f.per);
}

template <bool ROWS, bool WHOLE>
void launch_few_nk(const MatmulArgs& g, const FewPlan& f, float* part, hipStream_t st) {
  const dim3 grid((unsigned)f.groups, (unsigned)f.splits);
  if (f.nf == 1) fp8_matmul_few_kernel<false, ROWS, WHOLE, 1, 1><<<grid, 512, 0, st>>>(g, part, f.per);
  else launch_few_mf<false, ROWS, WHOLE, 2>(g, f, part, st);
}

template <bool WHOLE>
void launch_few(const MatmulArgs& g, float* ws, hipStream_t st) {
  const FewPlan f = few_plan(g);
  float* part = f.splits > 1 ? ws : nullptr;
  if (g.b_form == MOE_B_KN) launch_few_mf<true, false, WHOLE, 4>(g, f, part, st);
  else if (g.b_form == MOE_B_NK) launch_few_nk<false, WHOLE>(g, f, part, st);
  else launch_few_nk<true, WHOLE>(g, f, part, st);
  if (part)
    fp8_matmul_sum_kernel<WHOLE><<<(unsigned)((g.M * g.N / 4 + 255) / 256), 256, 0, st>>>(g, part, f.splits);
}

template <bool WHOLE>
void launch_tiles(const MatmulArgs& g, unsigned blocks, hipStream_t st) {
  if (g.b_form == MOE_B_KN) fp8_matmul_tile_kernel<MOE_B_KN, WHOLE><<<blocks, 256, 0, st>>>(g);
  else if (g.b_form == MOE_B_NK) fp8_matmul_tile_kernel<MOE_B_NK, WHOLE><<<blocks, 256, 0, st>>>(g);
  else fp8_matmul_tile_kernel<MOE_B_NK_ROWS, WHOLE><<<blocks, 256, 0, st>>>(g);
}

}  // namespace

size_t fp8_matmul_ws_bytes(const MatmulArgs& g) {
  if (g.M == 0 || g.M > kFewRows) return 0;
  const FewPlan f = few_plan(g);
  return f.splits > 1 ? (size_t)f.splits * g.M * g.N * sizeof(float) : 0;
}

hipError_t launch_fp8_matmul(const MatmulArgs& g, void* ws, hipStream_t st) {
  if (g.M <= kFewRows) {
    if (g.c_f32) launch_few<true>(g, (float*)ws, st);
    else launch_few<false>(g, (float*)ws, st);
    return hipGetLastError();
  }
  const unsigned blocks = (unsigned)((g.M + 127) / 128 * ((g.N + 127) / 128));
  if (g.c_f32) launch_tiles<true>(g, blocks, st);
  else launch_tiles<false>(g, blocks, st);
  return hipGetLastError();
}

}  // namespace moe
