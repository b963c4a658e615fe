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

// 8 consecutive values as they lie in memory, loaded once (non-temporal): a row's next loads are
// in flight as these while the row before is worked on.
template <bool F32>
struct Raw8 {
  u32x4_nt a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const u32x4_nt* q = (const u32x4_nt*)((const char*)p + i * (F32 ? 4 : 2));
    a = __builtin_nontemporal_load(q);
    if (F32) b = __builtin_nontemporal_load(q + 1);
  }
  __device__ __forceinline__ void zero() {
    a = u32x4_nt{0, 0, 0, 0};
    b = a;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (F32) x[j] = __uint_as_float(a[j]), x[4 + j] = __uint_as_float(b[j]);
      else x[2 * j] = lo_bf16(a[j]), x[2 * j + 1] = hi_bf16(a[j]);
    }
  }
};

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&x)[8]) {
  u32x4_nt* q = (u32x4_nt*)((char*)p + i * (F32 ? 4 : 2));
  if (F32) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      __builtin_nontemporal_store(u32x4_nt{__float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]),
                                           __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3])}, q + j);
  } else {
    __builtin_nontemporal_store(u32x4_nt{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                         pack_bf16x2(x[6], x[7])}, q);
  }
}

// 8 values of a weight or a gate (its type is the same for a whole launch), which other rows read too
__device__ __forceinline__ void load_w8(const void* p, int64_t i, bool f32, float (&x)[8]) {
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

__device__ __forceinline__ float load1(const void* p, int64_t i, bool f32) {
  return f32 ? ((const float*)p)[i] : bf16_to_f32(((const uint16_t*)p)[i]);
}

__device__ __forceinline__ void store1(void* p, int64_t i, bool f32, float x) {
  if (f32) ((float*)p)[i] = x;
  else ((uint16_t*)p)[i] = f32_to_bf16(x);
}

// A barrier that waits for LDS alone: global loads and stores stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Rows are spread over LR lanes of 8 values each, NV times: a part of a wave for short rows (heads), up
// to 16 waves for long ones.  A block holds the most rows that 1024 threads do (a power of two), and
// there is one block a compute unit.  Forward, while all rows fit the card at once: blocks of 256 threads
// or of one row, as many as hold them.
constexpr int norm_threads(int LR) { return 2 * LR > 1024 ? LR : LR % 192 == 0 ? 768 : 1024; }
constexpr int norm_few_threads(int LR) { return LR <= 128 ? 256 : LR; }

// The thread's row in its block; the same for a whole wave (and known to be, so that a row's addresses
// stay in scalar registers) but for rows on a part of a wave.
template <int LR>
__device__ __forceinline__ int row_slot() {
  const int s = threadIdx.x / LR;
  return LR >= 64 ? __builtin_amdgcn_readfirstlane(s) : s;
}

// First row of the block in a turn that starts at row `turn`.  Blocks go to the 8 XCDs one by one; in long
// batches' full turns each XCD takes rows side by side (backward, 16384 rows of 2048 in bf16: in the blocks'
// order 2 us more; 2048 rows, where it is kept: 0.9 us less.  Forward both are the same within 1 %).
__device__ __forceinline__ int64_t turn_row(int64_t turn, int64_t step, int64_t T, int rows) {
  const unsigned b = blockIdx.x, n = gridDim.x;
  const bool side = n % 8 == 0 && T >= 8 * step && turn + step <= T;
  return turn + (int64_t)(side ? b % 8 * (n / 8) + b / 8 : b) * rows;
}

// Sums of K values over a row's LR lanes, the same in every lane.  sh: [K][LR / 64] of the row and of
// this sum; the next sum takes another buffer, so that one barrier is enough (a wave that writes a
// buffer again has passed the barrier of the sum between, which every wave reaches after its reads of
// the first).  The block's rows reach it together.
template <int LR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* sh, int wave) {
#pragma unroll
  for (int q = 0; q < K; ++q) {
    if (LR >= 64) {
      v[q] = wave_sum_dpp(v[q]);
    } else {
      v[q] = row16_sum(v[q]);
      if (LR == 32) v[q] += __shfl_xor(v[q], 16, 64);
    }
  }
  if (LR > 64) {
    constexpr int W = LR / 64;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int q = 0; q < K; ++q) sh[q * W + wave] = v[q];
    lds_barrier();
#pragma unroll
    for (int q = 0; q < K; ++q) {
      v[q] = sh[q * W];
#pragma unroll
      for (int w = 1; w < W; ++w) v[q] += sh[q * W + w];
    }
  }
}

}  // namespace

// A block walks rows a grid apart, each row's loads issued before the row before is worked on; a row
// stays in registers between its passes, and so do the weights.  FEW: each block has its rows once, and
// loads the weights where it needs them, so that 64 registers do and a compute unit holds 2048 threads
// (rows of 2048 values, by one block a unit: 1 row 0.5 us more, 512 rows 0.8, 2048 rows 1.0; 4096 rows, which
// no longer fit, 0.6 less).  One row: 2.4 us.  Bound by HBM: 16384 rows of 2048 in bf16, both norms: 45 us,
// 5.9 TB/s (a block for each row 3 us more; cached loads and stores 6), with an fp32 stream 71 us, 5.7 TB/s;
// 64527 rows of 520: 50 us (a block for two rows 12 more); 3728 of 9000: 49 us (without the loads ahead 6
// more).
template <int LR, int NV, bool HF32, bool FEW>
__global__ __launch_bounds__(FEW ? norm_few_threads(LR) : norm_threads(LR), FEW && NV == 1 ? 8 : 1) void norm_forward_kernel(
    NormArgs p, const uint16_t* __restrict__ y, const void* h, const void* __restrict__ w_post,
    const void* __restrict__ gate, const void* __restrict__ w_pre, void* h_out, uint16_t* __restrict__ x) {
  constexpr int kRows = (FEW ? norm_few_threads(LR) : norm_threads(LR)) / LR, W = LR < 64 ? 1 : LR / 64;
  __shared__ float sh[kRows][2][W];
  const int slot = row_slot<LR>(), lane = threadIdx.x % LR, wave = lane >> 6;
  // the weights of a lane's columns: w_pre, and out_scale w_post with a channel's gate
  const auto load_pre = [&](int c, float (&v)[8]) { load_w8(w_pre, c, p.w_f32, v); };
  const auto load_post = [&](int c, float (&v)[8]) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p.out_scale;
    if (w_post) {
      load_w8(w_post, c, p.w_f32, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= w[i];
    }
    if (p.gate == G_CHANNEL) {
      load_w8(gate, c, p.w_f32, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= w[i];
    }
  };
  float wp[NV][8], cw[NV][8];
#pragma unroll
  for (int n = 0; n < NV && !FEW; ++n) {
    const int c = (n * LR + lane) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) wp[n][i] = cw[n][i] = 0.0f;
    if (c < p.d && x) load_pre(c, wp[n]);
    if (c < p.d && y) load_post(c, cw[n]);
  }
  const int64_t step = (int64_t)gridDim.x * kRows;
  Raw8<false> yr[NV];
  Raw8<HF32> hr[NV];
  float gt = 1.0f;
  const auto fetch = [&](int64_t t) {  // a row as it lies in memory
    gt = 1.0f;
    if (p.gate == G_TOKEN && t < p.T) gt = load1(gate, t, p.w_f32);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * LR + lane) * 8;
      hr[n].zero();
      yr[n].zero();
      if (t < p.T && c < p.d) {
        hr[n].load(h, t * p.d + c);
        if (y) yr[n].load(y, t * p.d + c);
      }
    }
  };
  fetch((int64_t)blockIdx.x * kRows + slot);
  int par = 0;  // the sums' two buffers in turn
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < p.T; t0 = FEW ? p.T : t0 + step) {
    const int64_t t = t0 + slot;
    const bool on = t < p.T;
    const int64_t base = on ? t * p.d : 0;
    float hv[NV][8], yv[NV][8];
#pragma unroll
    for (int n = 0; n < NV; ++n) hr[n].get(hv[n]), yr[n].get(yv[n]);
    float s[1] = {0.0f}, sq = gt;
    if (!FEW && t0 + step < p.T) fetch(t + step);
    if (y) {
      if (w_post) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] += yv[n][i] * yv[n][i];
        row_sum<LR, 1>(s, sh[slot][par], wave);
        par ^= 1;
        sq *= rsqrtf(s[0] * p.inv_d + p.eps);
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int c = (n * LR + lane) * 8;
        if (!on || c >= p.d) continue;
        if (FEW) load_post(c, cw[n]);
        if (p.gate == G_FULL) {
          float w[8];
          load_w8(gate, base + c, p.w_f32, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) yv[n][i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) hv[n][i] = p.res_scale * hv[n][i] + yv[n][i] * (cw[n][i] * sq);
        store8<HF32>(h_out, base + c, hv[n]);
      }
    }
    if (!x) continue;
    s[0] = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += hv[n][i] * hv[n][i];
    row_sum<LR, 1>(s, sh[slot][par], wave);
    par ^= 1;
    const float sp = rsqrtf(s[0] * p.inv_d + p.eps);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * LR + lane) * 8;
      if (!on || c >= p.d) continue;
      if (FEW) load_pre(c, wp[n]);
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = wp[n][i] * hv[n][i] * sp;
      store8<false>(x, base + c, w);
    }
  }
}

namespace {

// What one row of the backward pass reads, as it lies in memory
template <int NV, bool HF32, bool Y, bool P>
struct RowIn {
  float gt;  // the token's gate
  Raw8<HF32> h[NV], D[NV];
  Raw8<false> g[NV], y[NV];
};

}  // namespace

// A block walks rows a grid apart, each row's loads issued before the row before is worked on, and
// keeps the weights and the sums for their gradients of its columns in registers; the sums leave
// once, as partial sums that norm_reduce_kernel adds in a fixed order.
//
// With cwg = out_scale gate w_post of a channel (the token's gate apart, as gt), one sum serves the norm
// behind the block and a channel's gate: A = sum_t gt D yh gives dw_post = out_scale gate A and
// dgate = out_scale w_post A.
//
// Bound by HBM, 21 vector operations a value: 16384 rows of 2048 in bf16: 67 us, 6.1 TB/s with the partial
// sums, and 5 for norm_reduce_kernel; 4099 of 7168 with an fp32 stream: 101 us, 5.3 TB/s (17 turns of
// 256 blocks for 16.01 rows each).  Rows of more than 8192 values: a lane has 16, nothing is loaded ahead,
// and with both norms 28 of its 128 registers are spilled (41 to 45 with a gate for each value): 2048 rows
// of 16384 in bf16 127 us, 3.2 TB/s, 3728 of 9000 165 us; with one of the norms, which spills nothing, 54
// and 57 us, 5.0 and 4.7 TB/s.
template <int LR, int NV, bool HF32, bool Y, bool P, bool FULL>
__global__ __launch_bounds__(norm_threads(LR)) void norm_backward_kernel(
    NormArgs p, const uint16_t* __restrict__ y, const void* __restrict__ h_out, const void* __restrict__ w_post,
    const void* __restrict__ gate, const void* __restrict__ w_pre, const void* dh_out, const uint16_t* __restrict__ dx,
    void* dh, uint16_t* __restrict__ dy, void* __restrict__ dgate, float* __restrict__ part, int64_t part_stride) {
  constexpr int kRows = norm_threads(LR) / LR, W = LR < 64 ? 1 : LR / 64;
  __shared__ float sh[kRows][2][3 * W];
  const int slot = row_slot<LR>(), lane = threadIdx.x % LR, wave = lane >> 6;
  // the weights of a lane's columns: in registers, or for the longest rows in LDS (16 values a lane of each
  // would spill still more: 2048 rows of 16384 half as long again)
  constexpr bool kLds = NV > 1;
  __shared__ float4 w_lds[kLds ? 4 * NV * LR : 1];
  float a_pre[NV][8], a_post[NV][8], w_reg[NV][2][8];  // w_pre; out_scale gate w_post
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int c = (n * LR + lane) * 8;
    float wp[8], cwg[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a_pre[n][i] = a_post[n][i] = wp[i] = 0.0f, cwg[i] = FULL ? 1.0f : p.out_scale;
    if (c < p.d) {
      if (P) load_w8(w_pre, c, p.w_f32, wp);
      if (Y && w_post) {
        load_w8(w_post, c, p.w_f32, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) cwg[i] *= w[i];
      }
      if (Y && p.gate == G_CHANNEL) {
        load_w8(gate, c, p.w_f32, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) cwg[i] *= w[i];
      }
    }
    if (kLds) {  // a lane reads what it wrote itself
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        w_lds[(n * 4 + q) * LR + lane] = make_float4(wp[4 * q], wp[4 * q + 1], wp[4 * q + 2], wp[4 * q + 3]);
        w_lds[(n * 4 + 2 + q) * LR + lane] = make_float4(cwg[4 * q], cwg[4 * q + 1], cwg[4 * q + 2], cwg[4 * q + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w_reg[n][0][i] = wp[i], w_reg[n][1][i] = cwg[i];
    }
  }
  const auto weights = [&](int n, int which, float (&w)[8]) {
    if (kLds) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 v = w_lds[(n * 4 + 2 * which + q) * LR + lane];
        w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = w_reg[n][which][i];
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  RowIn<NV, HF32, Y, P> cur;
  const auto fetch = [&](int64_t t) {
    cur.gt = 1.0f;
    if (Y && p.gate == G_TOKEN && t < p.T) cur.gt = load1(gate, t, p.w_f32);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * LR + lane) * 8;
      const int64_t at = t * p.d + c;
      cur.D[n].zero();
      if (P) cur.h[n].zero(), cur.g[n].zero();
      if (Y) cur.y[n].zero();
      if (t < p.T && c < p.d) {
        if (dh_out) cur.D[n].load(dh_out, at);
        if (P) cur.h[n].load(h_out, at), cur.g[n].load(dx, at);
        if (Y) cur.y[n].load(y, at);
      }
    }
  };
  // a second row's values fit 128 registers beside the first's, but for the longest rows and a gate of its
  // own for each value beside the norm before a block (16384 x 2048: 95 us, loaded ahead and spilled 46 more)
  constexpr bool kAhead = NV == 1 && !(FULL && P);
  int64_t turn = 0, t0 = turn_row(0, step, p.T, kRows);
  if (kAhead) fetch(t0 + slot);
  int first = 0;  // the first sum's buffer: with one sum a row, two rows in turn
  while (t0 < p.T) {
    const int64_t t = t0 + slot;
    const bool on = t < p.T;
    turn += step;
    t0 = turn_row(turn, step, p.T, kRows);  // the next row
    const int64_t base = on ? t * p.d : 0;
    if (!Y) first ^= 1;
    if (!kAhead) fetch(t);
    const RowIn<NV, HF32, Y, P> in = cur;
    if (kAhead && t0 < p.T) fetch(t0 + slot);
    constexpr int kS = (P ? 2 : 0) + (Y ? 1 : 0);
    float s[kS];  // (h'^2, h' w_pre dx), (y^2)
#pragma unroll
    for (int q = 0; q < kS; ++q) s[q] = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if (P) {
        float h[8], g[8], w[8];
        in.h[n].get(h);
        in.g[n].get(g);
        weights(n, 0, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += h[i] * h[i], s[P ? 1 : 0] += h[i] * g[i] * w[i];
      }
      if (Y) {
        float v[8];
        in.y[n].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[kS - 1] += v[i] * v[i];
      }
    }
    row_sum<LR, kS>(s, sh[slot][first], wave);
    const float sp = P ? rsqrtf(s[0] * p.inv_d + p.eps) : 0.0f, mp = P ? s[1] * p.inv_d * sp * sp : 0.0f;
    const float sq = Y && w_post ? rsqrtf(s[kS - 1] * p.inv_d + p.eps) : 1.0f, sqg = sq * in.gt;
    float D[NV][8];
    float e[1] = {0.0f};  // D cwg y
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * LR + lane) * 8;
      in.D[n].get(D[n]);
      if (P) {
        float h[8], g[8], w[8];
        in.h[n].get(h);
        in.g[n].get(g);
        weights(n, 0, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[i] *= sp;
          a_pre[n][i] += h[i] * g[i];
          D[n][i] += w[i] * g[i] * sp;
          D[n][i] -= h[i] * mp;
        }
      }
      const bool in_row = on && c < p.d;
      if (dh && in_row) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = p.res_scale * D[n][i];
        store8<HF32>(dh, base + c, o);
      }
      if (Y) {
        float v[8], cwg[8];
        in.y[n].get(v);
        weights(n, 1, cwg);
        if (FULL) {
          // D: w_post' dn with the channel's own gate; the gate's gradient has the value itself
          float gv[8], dg[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) gv[i] = 0.0f;
          if (in_row) load_w8(gate, base + c, p.w_f32, gv);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float q = p.out_scale * D[n][i] * (v[i] * sq);
            dg[i] = q * cwg[i];
            a_post[n][i] += q * gv[i];
            e[0] += dg[i] * gv[i];
            D[n][i] *= p.out_scale * gv[i];
          }
          if (dgate && in_row) {
            if (p.w_f32) store8<true>(dgate, base + c, dg);
            else store8<false>(dgate, base + c, dg);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float q = D[n][i] * v[i];
            a_post[n][i] += q * sqg;
            e[0] += q * cwg[i];
          }
        }
      }
    }
    if (!Y) continue;
    row_sum<LR, 1>(e, sh[slot][1], wave);
    if (!FULL) e[0] *= sq;
    if (p.gate == G_TOKEN && dgate && on && lane == 0) store1(dgate, t, p.w_f32, e[0]);
    if (!dy) continue;
    const float mq = w_post ? e[0] * p.inv_d * sq : 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * LR + lane) * 8;
      if (!on || c >= p.d) continue;
      float v[8], cwg[8], o[8];
      in.y[n].get(v);
      weights(n, 1, cwg);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = sqg * (D[n][i] * cwg[i] - v[i] * mq);
      store8<false>(dy, base + c, o);
    }
  }
  if (!part) return;
  if (kRows == 1) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * LR + lane) * 8;
      if (c >= p.d) continue;
      if (P) store8<true>(part, (int64_t)blockIdx.x * p.d + c, a_pre[n]);
      if (Y) store8<true>(part, part_stride + (int64_t)blockIdx.x * p.d + c, a_post[n]);
    }
    return;
  }
  // the block's rows, in order (NV is 1 here)
  constexpr int kCols = kRows * LR * 8;
  __shared__ float red[kRows > 1 ? 2 * kCols : 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (P) red[slot * LR * 8 + lane * 8 + i] = a_pre[0][i];
    if (Y) red[kCols + slot * LR * 8 + lane * 8 + i] = a_post[0][i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.d; c += norm_threads(LR)) {
    float u = 0.0f, v = 0.0f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (P) u += red[r * LR * 8 + c];
      if (Y) v += red[kCols + r * LR * 8 + c];
    }
    if (P) part[(int64_t)blockIdx.x * p.d + c] = u;
    if (Y) part[part_stride + (int64_t)blockIdx.x * p.d + c] = v;
  }
}

// Sums over rows of the partial sums, 16 waves sharing the rows of 64 columns: of part[0] for dw_pre,
// of part[1] for dw_post and a channel gate's gradient (out_scale gate A and out_scale w_post A; where
// the rows' own gates are in the sum already, dw_post alone).
__global__ __launch_bounds__(1024) void norm_reduce_kernel(NormArgs p, const float* __restrict__ part,
                                                           int64_t part_stride, int rows, int first,
                                                           const void* w_post, const void* gate, void* dw_pre,
                                                           void* dw_post, void* dgate) {
  __shared__ float sh[16][64];
  const int which = first + blockIdx.y;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  const float* src = part + which * part_stride;
  float a = 0.0f;
  if (c < p.d) {
#pragma unroll 8
    for (int r = wv; r < rows; r += 16) a += src[(int64_t)r * p.d + c];
  }
  sh[wv][lane] = a;
  __syncthreads();
  if (wv != 0 || c >= p.d) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) a += sh[w][lane];
  if (which == 0) {
    store1(dw_pre, c, p.w_f32, a);
    return;
  }
  float by = p.gate == G_FULL ? 1.0f : p.out_scale;
  if (dgate) store1(dgate, c, p.w_f32, (w_post && rows ? load1(w_post, c, p.w_f32) : 1.0f) * p.out_scale * a);
  if (p.gate == G_CHANNEL && rows) by *= load1(gate, c, p.w_f32);
  if (dw_post) store1(dw_post, c, p.w_f32, by * a);
}

namespace {

// Lanes of a row of d values, the fewest that hold it 8 values each
int norm_lanes(int d) {
  for (const int lanes : {16, 32, 64, 128, 192, 256, 384, 512, 768})
    if (d <= 8 * lanes) return lanes;
  return 1024;
}

#define MOE_NORM_DISPATCH(d, CALL)                 \
  do {                                             \
    switch (norm_lanes(d)) {                       \
      case 16: { CALL(16, 1); } break;             \
      case 32: { CALL(32, 1); } break;             \
      case 64: { CALL(64, 1); } break;             \
      case 128: { CALL(128, 1); } break;           \
      case 192: { CALL(192, 1); } break;           \
      case 256: { CALL(256, 1); } break;           \
      case 384: { CALL(384, 1); } break;           \
      case 512: { CALL(512, 1); } break;           \
      case 768: { CALL(768, 1); } break;           \
      default:                                     \
        if ((d) <= 8 * 1024) { CALL(1024, 1); }    \
        else { CALL(1024, 2); }                    \
    }                                              \
  } while (0)

// One block a compute unit, each with its rows' loads ahead.  Smaller blocks, more of them, write more
// partial sums and read memory in smaller pieces (backward, 16384 rows of 2048 values, beside one block of four
// rows a unit: 2 blocks of one row 5 us more, 4 of them 12, 1 block of two rows 2).
int norm_blocks(int64_t T, int d) {
  const int rows = norm_threads(norm_lanes(d)) / norm_lanes(d);
  const int64_t b = (T + rows - 1) / rows;
  return (int)(b < 256 ? b : 256);
}

}  // namespace

size_t norm_ws_bytes(int64_t T, int d) {
  return (size_t)(2 * (int64_t)norm_blocks(T, d) * d * 4);
}

hipError_t launch_norm_forward(const NormArgs& p, const uint16_t* y, const void* h, const void* w_post,
                               const void* gate, const void* w_pre, void* h_out, uint16_t* x, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  const int lanes = norm_lanes(p.d), few_rows = norm_few_threads(lanes) / lanes;
  const bool few = p.T <= 256 * 2048 / lanes;  // lanes that the card holds
  const int blocks = few ? (int)((p.T + few_rows - 1) / few_rows) : norm_blocks(p.T, p.d);
#define MOE_NORM_LAUNCH(LR, NV, F, FEW)                                                                \
  norm_forward_kernel<LR, NV, F, FEW><<<blocks, FEW ? norm_few_threads(LR) : norm_threads(LR), 0, st>>>( \
      p, y, h, w_post, gate, w_pre, h_out, x)
#define MOE_NORM_CALL(LR, NV)                             \
  if (few && p.h_f32) MOE_NORM_LAUNCH(LR, NV, true, true); \
  else if (few) MOE_NORM_LAUNCH(LR, NV, false, true);      \
  else if (p.h_f32) MOE_NORM_LAUNCH(LR, NV, true, false);  \
  else MOE_NORM_LAUNCH(LR, NV, false, false)
  MOE_NORM_DISPATCH(p.d, MOE_NORM_CALL);
#undef MOE_NORM_CALL
#undef MOE_NORM_LAUNCH
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& p, const uint16_t* y, const void* h_out, const void* w_post,
                                const void* gate, const void* w_pre, const void* dh_out, const uint16_t* dx, void* dh,
                                uint16_t* dy, void* dw_post, void* dgate, void* dw_pre, float* part, hipStream_t st) {
  const int blocks = norm_blocks(p.T, p.d);
  const int64_t stride = (int64_t)blocks * p.d;
  void* dg = p.gate == G_CHANNEL ? dgate : nullptr;
  const bool pre = dw_pre, post = dw_post || dg;
  if (p.T > 0) {
    const bool full = y && p.gate == G_FULL;
#define MOE_NORM_RUN(LR, NV, H, Y, P, F)                                                                              \
  norm_backward_kernel<LR, NV, H, Y, P, F><<<blocks, norm_threads(LR), 0, st>>>(p, y, h_out, w_post, gate, w_pre, dh_out, \
                                                                              dx, dh, dy, dgate,                       \
                                                                              pre || post ? part : nullptr, stride)
#define MOE_NORM_FORM(LR, NV, H)                                 \
  if (!y) MOE_NORM_RUN(LR, NV, H, false, true, false);           \
  else if (w_pre && full) MOE_NORM_RUN(LR, NV, H, true, true, true); \
  else if (w_pre) MOE_NORM_RUN(LR, NV, H, true, true, false);    \
  else if (full) MOE_NORM_RUN(LR, NV, H, true, false, true);     \
  else MOE_NORM_RUN(LR, NV, H, true, false, false)
#define MOE_NORM_CALL(LR, NV)                   \
  if (p.h_f32) { MOE_NORM_FORM(LR, NV, true); } \
  else { MOE_NORM_FORM(LR, NV, false); }
    MOE_NORM_DISPATCH(p.d, MOE_NORM_CALL);
#undef MOE_NORM_CALL
#undef MOE_NORM_FORM
#undef MOE_NORM_RUN
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (pre || post)
    norm_reduce_kernel<<<dim3((p.d + 63) / 64, pre && post ? 2 : 1), 1024, 0, st>>>(
        p, part, stride, p.T > 0 ? blocks : 0, pre ? 0 : 1, w_post, gate, dw_pre, dw_post, dg);
  return hipGetLastError();
}

}  // namespace moe
