// RMS norms before and after a block, with the block's gate and the scaled residual, and their
// gradients.  One row is a token's d values:
//   n = w_post * y / rms(y)  (y itself without w_post)      rms(v) = sqrt(mean v^2 + eps)
//   h' = res_scale h + out_scale gate n                      x = w_pre * h' / rms(h')
// Backward, from dh' and dx, with s_p = 1/rms(h'), hh = h' s_p, s_q = 1/rms(y), yh = y s_q:
//   D = dh' + s_p (w_pre dx - hh mean(hh w_pre dx))          dh = res_scale D
//   dw_pre = sum_t dx hh                                     dgate = out_scale D n (summed)
//   dn = out_scale gate D,  dw_post = sum_t dn yh,  dy = s_q (w_post dn - yh mean(yh w_post dn))
// The routed layer sits between the two norms (page "NVIDIA מציגה דרך יעילה לאמן מודלי MoE
// בביולוגיה": transformer blocks whose feed-forward part is the expert layer).
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

enum { G_NONE = 0, G_CHANNEL = 1, G_TOKEN = 2, G_FULL = 3 };

// 8 consecutive values of an array in fp32 or bf16, from element i (a multiple of 8)
__device__ __forceinline__ void load8(const void* p, int64_t i, bool f32, float (&x)[8]) {
  if (f32) {
    const float4 a = ((const float4*)((const float*)p + i))[0], b = ((const float4*)((const float*)p + i))[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 w = *(const uint4*)((const uint16_t*)p + i);
    x[0] = lo_bf16(w.x), x[1] = hi_bf16(w.x), x[2] = lo_bf16(w.y), x[3] = hi_bf16(w.y);
    x[4] = lo_bf16(w.z), x[5] = hi_bf16(w.z), x[6] = lo_bf16(w.w), x[7] = hi_bf16(w.w);
  }
}

__device__ __forceinline__ void store8(void* p, int64_t i, bool f32, const float (&x)[8]) {
  if (f32) {
    float4* o = (float4*)((float*)p + i);
    o[0] = make_float4(x[0], x[1], x[2], x[3]);
    o[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *(uint4*)((uint16_t*)p + i) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                             pack_bf16x2(x[6], x[7]));
  }
}

__device__ __forceinline__ float load1(const void* p, int64_t i, bool f32) {
  return f32 ? ((const float*)p)[i] : bf16_to_f32(((const uint16_t*)p)[i]);
}

__device__ __forceinline__ void store1(void* p, int64_t i, bool f32, float x) {
  if (f32) ((float*)p)[i] = x;
  else ((uint16_t*)p)[i] = f32_to_bf16(x);
}

// Sums of K values over a row's W waves, in the same order for every lane.  sh: [K][W] of the row;
// the block's rows reach it together.
template <int W, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* sh, int wave) {
#pragma unroll
  for (int q = 0; q < K; ++q)
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v[q] += __shfl_xor(v[q], m, 64);
  if (W > 1) {
    __syncthreads();  // the last sums have been read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int q = 0; q < K; ++q) sh[q * W + wave] = v[q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < K; ++q) {
      v[q] = sh[q * W];
#pragma unroll
      for (int w = 1; w < W; ++w) v[q] += sh[q * W + w];
    }
  }
}

// W waves a row, NV times 8 values a lane: the row stays in registers between its passes.
template <int W, int NV>
__global__ __launch_bounds__(W <= 4 ? 256 : 512) void norm_forward_kernel(NormArgs p, const uint16_t* __restrict__ y,
                                                                         const void* h, const void* __restrict__ w_post,
                                                                         const void* __restrict__ gate,
                                                                         const void* __restrict__ w_pre, void* h_out,
                                                                         uint16_t* __restrict__ x) {
  constexpr int kRows = W <= 4 ? 4 / W : 1;
  __shared__ float sh[kRows][2 * W];
  const int slot = threadIdx.x / (64 * W), lane = threadIdx.x % (64 * W), wave = lane >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRows + slot;
  const bool on = t < p.T;
  const int64_t base = on ? t * p.d : 0;
  float yv[NV][8], hv[NV][8];
  float s[1] = {0.0f};
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int c = (n * 64 * W + lane) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) yv[n][i] = 0.0f, hv[n][i] = 0.0f;
    if (on && c < p.d) {
      load8(h, base + c, p.h_f32, hv[n]);
      if (y) load8(y, base + c, false, yv[n]);
    }
  }
  if (y) {
    float sq = 1.0f;
    if (w_post) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += yv[n][i] * yv[n][i];
      row_sum<W, 1>(s, sh[slot], wave);
      sq = rsqrtf(s[0] * p.inv_d + p.eps);
    }
    sq *= p.out_scale;
    if (p.gate == G_TOKEN && on) sq *= load1(gate, t, p.w_f32);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * 64 * W + lane) * 8;
      if (!on || c >= p.d) continue;
      float m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = sq;
      if (w_post) {
        float w[8];
        load8(w_post, c, p.w_f32, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] *= w[i];
      }
      if (p.gate == G_CHANNEL || p.gate == G_FULL) {
        float w[8];
        load8(gate, p.gate == G_FULL ? base + c : c, p.w_f32, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] *= w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) hv[n][i] = p.res_scale * hv[n][i] + yv[n][i] * m[i];
      store8(h_out, base + c, p.h_f32, hv[n]);
    }
  }
  if (!x) return;
  s[0] = 0.0f;
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += hv[n][i] * hv[n][i];
  row_sum<W, 1>(s, sh[slot], wave);
  const float sp = rsqrtf(s[0] * p.inv_d + p.eps);
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int c = (n * 64 * W + lane) * 8;
    if (!on || c >= p.d) continue;
    float w[8];
    load8(w_pre, c, p.w_f32, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] *= hv[n][i] * sp;
    store8(x, base + c, false, w);
  }
}

// A block walks rows a grid apart and keeps the weights' gradients of its columns in registers;
// they leave once, as partial sums that norm_reduce_kernel adds in a fixed order.
template <int W, int NV>
__global__ __launch_bounds__(W <= 4 ? 256 : 512) void norm_backward_kernel(
    NormArgs p, const uint16_t* __restrict__ y, const void* __restrict__ h_out, const void* __restrict__ w_post,
    const void* __restrict__ gate, const void* __restrict__ w_pre, const void* dh_out, const uint16_t* __restrict__ dx,
    void* dh, uint16_t* __restrict__ dy, void* __restrict__ dgate, float* __restrict__ part, int64_t part_stride) {
  constexpr int kRows = W <= 4 ? 4 / W : 1;
  __shared__ float sh[kRows][4 * W];
  const int slot = threadIdx.x / (64 * W), lane = threadIdx.x % (64 * W), wave = lane >> 6;
  float a_pre[NV][8], a_post[NV][8], a_gate[NV][8];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) a_pre[n][i] = a_post[n][i] = a_gate[n][i] = 0.0f;
  const bool each = p.gate == G_CHANNEL || p.gate == G_FULL;  // a gate value of its own for each channel
  const int64_t step = (int64_t)gridDim.x * kRows;
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < p.T; t0 += step) {
    const int64_t t = t0 + slot;
    const bool on = t < p.T;
    const int64_t base = on ? t * p.d : 0;
    float D[NV][8], hv[NV][8], yv[NV][8];
    float s[3] = {0.0f, 0.0f, 0.0f};  // h'^2, h' w_pre dx, y^2
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * 64 * W + lane) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) D[n][i] = hv[n][i] = yv[n][i] = 0.0f;
      if (!on || c >= p.d) continue;
      if (dh_out) load8(dh_out, base + c, p.h_f32, D[n]);
      if (w_post) {
        load8(y, base + c, false, yv[n]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] += yv[n][i] * yv[n][i];
      }
      if (w_pre) {
        float w[8], g[8];
        load8(h_out, base + c, p.h_f32, hv[n]);
        load8(dx, base + c, false, g);
        load8(w_pre, c, p.w_f32, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += hv[n][i] * hv[n][i], s[1] += hv[n][i] * (w[i] * g[i]);
      }
    }
    row_sum<W, 3>(s, sh[slot], wave);
    const float sp = rsqrtf(s[0] * p.inv_d + p.eps), sq = w_post ? rsqrtf(s[2] * p.inv_d + p.eps) : 1.0f;
    const float mp = s[1] * p.inv_d * sp * sp * sp;
    float gt = p.out_scale;
    if (p.gate == G_TOKEN && on) gt *= load1(gate, t, p.w_f32);
    float e[2] = {0.0f, 0.0f};  // y w_post gate D (or without the token's gate), for dy's mean and a token's dgate
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * 64 * W + lane) * 8;
      if (!on || c >= p.d) continue;
      if (w_pre) {
        float w[8], g[8];
        load8(dx, base + c, false, g);
        load8(w_pre, c, p.w_f32, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a_pre[n][i] += g[i] * (hv[n][i] * sp);
          D[n][i] += sp * (w[i] * g[i]) - hv[n][i] * mp;
        }
      }
      if (dh) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = p.res_scale * D[n][i];
        store8(dh, base + c, p.h_f32, o);
      }
      if (!y) continue;
      // hv: now gate * out_scale of each channel;  D: dn = out_scale gate D
      if (!w_post) load8(y, base + c, false, yv[n]);
      float w[8], gv[8], dg[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f, gv[i] = gt;
      if (w_post) load8(w_post, c, p.w_f32, w);
      if (each) {
        load8(gate, p.gate == G_FULL ? base + c : c, p.w_f32, gv);
#pragma unroll
        for (int i = 0; i < 8; ++i) gv[i] *= p.out_scale;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yh = yv[n][i] * sq;
        dg[i] = p.out_scale * D[n][i] * (w[i] * yh);
        e[1] += dg[i];
        D[n][i] *= gv[i];
        a_post[n][i] += D[n][i] * yh;
        D[n][i] *= w[i];
        e[0] += D[n][i] * yh;
        a_gate[n][i] += dg[i];
      }
      if (p.gate == G_FULL && dgate) store8(dgate, base + c, p.w_f32, dg);
    }
    if (!y) continue;
    row_sum<W, 2>(e, sh[slot], wave);
    if (p.gate == G_TOKEN && dgate && on && lane == 0) store1(dgate, t, p.w_f32, e[1]);
    if (!dy) continue;
    const float mq = w_post ? e[0] * p.inv_d * sq : 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * 64 * W + lane) * 8;
      if (!on || c >= p.d) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = sq * (D[n][i] - yv[n][i] * mq);
      store8(dy, base + c, false, o);
    }
  }
  if (!part) return;
  const int64_t row = (int64_t)blockIdx.x * kRows + slot;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int c = (n * 64 * W + lane) * 8;
    if (c >= p.d) continue;
    store8(part, row * p.d + c, true, a_pre[n]);
    store8(part, part_stride + row * p.d + c, true, a_post[n]);
    if (p.gate == G_CHANNEL) store8(part, 2 * part_stride + row * p.d + c, true, a_gate[n]);
  }
}

// out[q][c] = sum over rows of part[q][row][c]: 16 waves share the rows of 64 columns.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* __restrict__ part, int64_t part_stride, int rows,
                                                           int d, bool f32, void* o0, void* o1, void* o2) {
  __shared__ float sh[16][64];
  void* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  const float* src = part + (int64_t)blockIdx.y * part_stride;
  float a = 0.0f;
#pragma unroll 8
  for (int r = wv; r < rows; r += 16)
    if (c < d) a += src[(int64_t)r * d + c];
  sh[wv][lane] = a;
  __syncthreads();
  if (wv == 0 && c < d) {
#pragma unroll
    for (int w = 1; w < 16; ++w) a += sh[w][lane];
    store1(out, c, f32, a);
  }
}

// waves a row and 8-value vectors a lane for rows of d values
#define MOE_NORM_DISPATCH(d, CALL)          \
  do {                                      \
    if ((d) <= 512) { CALL(1, 1); }         \
    else if ((d) <= 1024) { CALL(2, 1); }   \
    else if ((d) <= 2048) { CALL(4, 1); }   \
    else if ((d) <= 4096) { CALL(4, 2); }   \
    else if ((d) <= 8192) { CALL(4, 4); }   \
    else { CALL(8, 4); }                    \
  } while (0)

int norm_rows_per_block(int d) { return d <= 512 ? 4 : d <= 1024 ? 2 : 1; }

int norm_bwd_blocks(int64_t T, int d) {
  const int64_t b = (T + norm_rows_per_block(d) - 1) / norm_rows_per_block(d);
  return (int)(b < 1024 ? b : 1024);
}

}  // namespace

size_t norm_ws_bytes(int64_t T, int d, int gate) {
  const int64_t rows = (int64_t)norm_bwd_blocks(T, d) * norm_rows_per_block(d);
  return (size_t)((gate == G_CHANNEL ? 3 : 2) * rows * d * 4);
}

hipError_t launch_norm_forward(const NormArgs& p, const uint16_t* y, const void* h, const void* w_post,
                               const void* gate, const void* w_pre, void* h_out, uint16_t* x, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  const unsigned blocks = (unsigned)((p.T + norm_rows_per_block(p.d) - 1) / norm_rows_per_block(p.d));
#define MOE_NORM_CALL(W, NV) \
  norm_forward_kernel<W, NV><<<blocks, W <= 4 ? 256 : 512, 0, st>>>(p, y, h, w_post, gate, w_pre, h_out, x)
  MOE_NORM_DISPATCH(p.d, MOE_NORM_CALL);
#undef MOE_NORM_CALL
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& p, const uint16_t* y, const void* h_out, const void* w_post,
                                const void* gate, const void* w_pre, const void* dh_out, const uint16_t* dx, void* dh,
                                uint16_t* dy, void* dw_post, void* dgate, void* dw_pre, float* part, hipStream_t st) {
  const int blocks = norm_bwd_blocks(p.T, p.d);
  const int rows = blocks * norm_rows_per_block(p.d);
  const int64_t stride = (int64_t)rows * p.d;
  void* dg = p.gate == G_CHANNEL ? dgate : nullptr;
  const bool sums = dw_pre || dw_post || dg;
  if (p.T > 0) {
#define MOE_NORM_CALL(W, NV)                                                                                      \
  norm_backward_kernel<W, NV><<<blocks, W <= 4 ? 256 : 512, 0, st>>>(p, y, h_out, w_post, gate, w_pre, dh_out, dx, \
                                                                     dh, dy, dgate, sums ? part : nullptr, stride)
    MOE_NORM_DISPATCH(p.d, MOE_NORM_CALL);
#undef MOE_NORM_CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (sums)
    norm_reduce_kernel<<<dim3((p.d + 63) / 64, 3), 1024, 0, st>>>(part, stride, p.T > 0 ? rows : 0, p.d, p.w_f32,
                                                                  dw_pre, dw_post, dg);
  return hipGetLastError();
}

}  // namespace moe
