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
    auto wide = [](const i32x8& v, int s) __attribute__((always_inline)) {
      bf16x8_t w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x2_t p = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * s + i / 2], 1.0f, true)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * s + i / 2], 1.0f, false);
        w[2 * i] = p[0];
        w[2 * i + 1] = p[1];
      }
      return w;
    };
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wide(b, s), wide(a, s), c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 0, 0, 0, 127, 0, 127);
  }
}

}  // namespace

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
        const int64_t at = row * g.ldc + col;
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] = acc[i][j][r + q];
          if (g.C_in) v[q] += g.c_f32 ? ((const float*)g.C_in)[at + q] : bf16_to_f32(((const uint16_t*)g.C_in)[at + q]);
        }
        if (g.c_f32) *(float4*)((float*)g.C + at) = make_float4(v[0], v[1], v[2], v[3]);
        else *(u32x2*)((uint16_t*)g.C + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
  }
}

size_t fp8_matmul_ws_bytes(const MatmulArgs&) { return 0; }

namespace {
template <bool WHOLE>
void launch_tiles(const MatmulArgs& g, unsigned blocks, hipStream_t st) {
  if (g.b_form == MOE_B_KN) fp8_matmul_tile_kernel<MOE_B_KN, WHOLE><<<blocks, 256, 0, st>>>(g);
  else if (g.b_form == MOE_B_NK) fp8_matmul_tile_kernel<MOE_B_NK, WHOLE><<<blocks, 256, 0, st>>>(g);
  else fp8_matmul_tile_kernel<MOE_B_NK_ROWS, WHOLE><<<blocks, 256, 0, st>>>(g);
}
}  // namespace

hipError_t launch_fp8_matmul(const MatmulArgs& g, void*, hipStream_t st) {
  const unsigned blocks = (unsigned)((g.M + 127) / 128 * ((g.N + 127) / 128));
  if (g.c_f32) launch_tiles<true>(g, blocks, st);
  else launch_tiles<false>(g, blocks, st);
  return hipGetLastError();
}

}  // namespace moe
