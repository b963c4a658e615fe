// Blockwise e4m3 quantisation: one fp32 scale (largest magnitude / 448) for 128 values of a row, for
// 128 rows of a column (written transposed, an operand of a product over the rows) or for 128 x 128.
// By rows the codes and scales are bit for bit those that the layer's fp8 path makes of dy, but in two cases: the
// layer saturates a NaN to -448 where this keeps it, and its scales follow a block's largest magnitude
// below 448 * 2^-126 too, past fp32's normal range.  ("NVIDIA מציגה דרך יעילה לאמן
// מודלי MoE בביולוגיה", section "צמצום הזיכרון ותקורות הכימות": quantisation adds work on top of the
// 16-bit master weights.)
//
// Every kernel reads its source once, 16 bytes a lane, keeps the values in registers between the
// maximum and the codes, and is bound by HBM.
#include "common.hpp"
#include "gemm_common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// Below this a block's scale would leave fp32's normal range.
constexpr float kLeastMax = 448.0f * 0x1p-126f;

struct Scale {
  float scale, factor;  // largest magnitude / 448 and its inverse
};
__device__ __forceinline__ Scale scale_of(float m) {
  const float c = fmaxf(m, kLeastMax);
  return m > 0.0f ? Scale{c / 448.0f, 448.0f / c} : Scale{1.0f, 1.0f};
}

// Four e4m3 codes; magnitudes past 448 (a factor's rounding) saturate, NaN stays NaN.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  auto sat = [](float v) { return v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v; };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), w, true);
  return (uint32_t)w;
}

// 8 neighbouring values of a row
template <bool F32>
__device__ __forceinline__ void load8(const void* src, int64_t at, float (&v)[8]) {
  if constexpr (F32) {
    const uint4 a = load_once16((const float*)src + at), b = load_once16((const float*)src + at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(word_of(a, i));
      v[4 + i] = __uint_as_float(word_of(b, i));
    }
  } else {
    const uint4 a = load_once16((const uint16_t*)src + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = lo_bf16(word_of(a, i));
      v[2 * i + 1] = hi_bf16(word_of(a, i));
    }
  }
}

__device__ __forceinline__ float max8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

}  // namespace

// 16 lanes for a block of 128 values of a row.
template <bool F32>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* __restrict__ src, int64_t ld, int64_t blocks,
                                                            int cols, int nb, uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
  const int64_t b = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
  if (b >= blocks) return;  // uniform over the block's 16 lanes
  const int64_t row = b / nb;
  const int col = (int)(b - row * nb) * 128 + (threadIdx.x % 16) * 8;
  const bool in = col < cols;
  float v[8] = {};
  if (in) load8<F32>(src, row * ld + col, v);
  const Scale s = scale_of(row16_max(max8(v)));
  if (in)
    *(u32x2*)(codes + row * cols + col) =
        u32x2{codes4(v[0] * s.factor, v[1] * s.factor, v[2] * s.factor, v[3] * s.factor),
              codes4(v[4] * s.factor, v[5] * s.factor, v[6] * s.factor, v[7] * s.factor)};
  if (threadIdx.x % 16 == 0) scales[b] = s.scale;
}

// 128 rows x 64 columns a block: thread (r, c) of 32 x 8 holds rows 4r .. 4r+3 of columns 8c .. 8c+7, so
// that a column's four codes are one word of the transposed row.  LDS keeps a column's words with their
// 16-byte pieces exchanged by the column's thread (8 c + j: piece ^ c), without which four lanes of a store
// meet in a bank.
// The rows of codes are padded to 16 tokens only, so that neighbouring blocks along the tokens share lines of
// 128 bytes: thread blocks are dealt out to the eight L2 caches so that each has a run of neighbours, and a line
// leaves its cache whole (21804x4096 bf16 79 -> 62 us; 4.4 TB/s, a copy 5.1).
template <bool F32>
__global__ __launch_bounds__(256) void quantize_tokens_kernel(const void* __restrict__ src, int64_t ld, int64_t rows,
                                                              int cols, int64_t r16, int64_t nb, int64_t tiles,
                                                              uint8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int LD = 36;  // words of a column in LDS: 32 and padding that keeps 16-byte rows
  __shared__ float sh_max[4][64];
  __shared__ __attribute__((aligned(16))) uint32_t sh[64 * LD];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t each = gridDim.x / 8, tile = blockIdx.x % 8 * each + blockIdx.x / 8;
  if (tile >= tiles) return;
  const int64_t tb = tile % nb;
  const int c0 = (int)(tile / nb) * 64, cc = tid % 8, rr = tid / 8;
  const int col = c0 + 8 * cc;
  float v[4][8] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = tb * 128 + 4 * rr + i;
    if (row < rows && col < cols) load8<F32>(src, row * ld + col, v[i]);
  }
  float m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = fmaxf(fmaxf(fabsf(v[0][j]), fabsf(v[1][j])), fmaxf(fabsf(v[2][j]), fabsf(v[3][j])));
#pragma unroll
    for (int x = 8; x < 64; x <<= 1) m[j] = fmaxf(m[j], __shfl_xor(m[j], x, 64));
  }
  if (lane < 8)
#pragma unroll
    for (int j = 0; j < 8; ++j) sh_max[wv][8 * lane + j] = m[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = 8 * cc + j;
    const Scale s = scale_of(fmaxf(fmaxf(sh_max[0][c], sh_max[1][c]), fmaxf(sh_max[2][c], sh_max[3][c])));
    sh[c * LD + (rr / 4 ^ cc) * 4 + rr % 4] = codes4(v[0][j] * s.factor, v[1][j] * s.factor, v[2][j] * s.factor, v[3][j] * s.factor);
    if (rr == 0 && col < cols) scales[(int64_t)(col + j) * nb + tb] = s.scale;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = (tid + 256 * i) / 8, q = tid % 8;
    const int64_t at = tb * 128 + 16 * q;
    if (c0 + c < cols && at < r16) *(uint4*)(codes + (c0 + c) * r16 + at) = *(const uint4*)&sh[c * LD + 4 * (q ^ (c / 8 & 7))];
  }
}

// A block of 128 x 128 a thread block; thread (r, c) of 16 x 16 holds rows r, r + 16, ... of 8 columns.
template <bool F32>
__global__ __launch_bounds__(256) void quantize_tiles_kernel(const void* __restrict__ src, int64_t ld, int64_t rows,
                                                             int cols, int nb, uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
  __shared__ float sh_max[4];
  const int tid = threadIdx.x;
  const int64_t tb = blockIdx.x / nb;
  const int cb = (int)(blockIdx.x - tb * nb);
  const int col = cb * 128 + 8 * (tid % 16);
  float v[8][8] = {}, m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = tb * 128 + tid / 16 + 16 * i;
    if (row < rows && col < cols) load8<F32>(src, row * ld + col, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, max8(v[i]));
  m = wave_max_dpp(m);
  if ((tid & 63) == 0) sh_max[tid >> 6] = m;
  __syncthreads();
  const Scale s = scale_of(fmaxf(fmaxf(sh_max[0], sh_max[1]), fmaxf(sh_max[2], sh_max[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = tb * 128 + tid / 16 + 16 * i;
    if (row < rows && col < cols)
      *(u32x2*)(codes + row * cols + col) =
          u32x2{codes4(v[i][0] * s.factor, v[i][1] * s.factor, v[i][2] * s.factor, v[i][3] * s.factor),
                codes4(v[i][4] * s.factor, v[i][5] * s.factor, v[i][6] * s.factor, v[i][7] * s.factor)};
  }
  if (tid == 0) scales[blockIdx.x] = s.scale;
}

namespace {
template <bool F32>
hipError_t quantize(const void* src, int64_t rows, int64_t cols, int64_t ld, int form, uint8_t* codes, float* scales,
                    hipStream_t st) {
  const int nb = (int)((cols + 127) / 128);
  const int64_t rb = (rows + 127) / 128;
  if (form == MOE_BLOCK_ROWS) {
    const int64_t blocks = rows * nb;
    quantize_rows_kernel<F32><<<(unsigned)((blocks + 15) / 16), 256, 0, st>>>(src, ld, blocks, (int)cols, nb, codes, scales);
  } else if (form == MOE_BLOCK_TOKENS) {
    const int64_t tiles = rb * ((cols + 63) / 64);
    quantize_tokens_kernel<F32><<<(unsigned)((tiles + 7) / 8 * 8), 256, 0, st>>>(src, ld, rows, (int)cols, (rows + 15) / 16 * 16, rb,
                                                                            tiles, codes, scales);
  } else {
    quantize_tiles_kernel<F32><<<(unsigned)(rb * nb), 256, 0, st>>>(src, ld, rows, (int)cols, nb, codes, scales);
  }
  return hipGetLastError();
}
}  // namespace

hipError_t launch_fp8_quantize(const void* src, bool f32, int64_t rows, int64_t cols, int64_t ld, int form,
                               uint8_t* codes, float* scales, hipStream_t st) {
  return f32 ? quantize<true>(src, rows, cols, ld, form, codes, scales, st)
             : quantize<false>(src, rows, cols, ld, form, codes, scales, st);
}

}  // namespace moe
