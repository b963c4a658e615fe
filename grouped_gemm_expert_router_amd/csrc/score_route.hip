// Routing by scores: softmax or sigmoid scores, a bias for balance, groups of experts, top-k and the
// weights of the chosen, with the weights' gradient and the bias's step.
//
// The choice: c = score + bias; of the groups (neighbouring experts) those with the largest sum of
// their one or two best c stay; of their experts the k largest c are taken, in descending order.
// Two c that differ by less than fp32 resolves are neighbours often enough in a batch (16384 tokens,
// eight choices each) that the order is taken from 64 bits.
//
// A learned router scores the experts and activates the top K (page "Az NVIDIA szerint tízszer
// gyorsabb lett a dropless MoE tanítása JAX-ban", section "A dropless MoE minden tokent feldolgoz");
// the bias acts against the uneven loads of its section "Az egyenetlen terhelés lassítja a tanítást".
#include <math.h>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// Blocks of four waves, a token each, that walk the tokens behind (a launch holds at most 2^32 threads).
unsigned token_grid(int T) { return (unsigned)(T < (1 << 24) ? (T + 3) / 4 : 1 << 22); }

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmax(v, __shfl_xor(v, m, 64));
  return v;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// e^(min(l, 0) - m) / (1 + e^-|l|): the sigmoid of l times e^-m, without overflow at any l
__device__ __forceinline__ double sigmoid_scaled(double l, double m) {
  return exp(fmin(l, 0.0) - m) / (1.0 + exp(-fabs(l)));
}

// Weights of a token's chosen experts, before `scale`: lane j < k holds slot j's logit l (there: the
// slot has an expert).  top, sum: maximum and sum of exponentials over all of the token's logits,
// for a softmax that is not renormalised.  Renormalised weights are quotients with the largest
// chosen logit taken out, so that they stay finite where every chosen score underflows.
__device__ __forceinline__ double chosen_weight(const ScoreArgs& p, bool there, double l, double top, double sum) {
  double z;
  if (p.sigmoid) {
    const double m = p.renorm ? wave_max_f64(there ? fmin(l, 0.0) : -INFINITY) : 0.0;
    z = there ? sigmoid_scaled(l, m) : 0.0;
  } else {
    const double m = p.renorm ? wave_max_f64(there ? l : -INFINITY) : top;
    z = there ? exp(l - m) : 0.0;
  }
  if (p.renorm) sum = wave_sum_f64(z);
  else if (p.sigmoid) sum = 1.0;
  return there ? z / sum : 0.0;
}

}  // namespace

// One wave per token; lane l holds the experts l, l + 64, ...  Everything in 64 bits.
template <int EPL>
__device__ __forceinline__ void score_choose_token(const ScoreArgs& p, const float* __restrict__ row,
                                                   const float* __restrict__ bias, bool masked, double* sh, int32_t* ids,
                                                   float* w) {
  const int lane = threadIdx.x & 63;
  if (masked) {
    if (lane < p.k) {
      ids[lane] = -1;
      w[lane] = 0.0f;
    }
    return;
  }
  float x[EPL];
  float xmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < p.E ? row[e] : -INFINITY;
    xmax = fmaxf(xmax, x[i]);
  }
  double top = 0.0, sum = 1.0, c[EPL];
  if (!p.sigmoid) {
    top = wave_max_f64(xmax);
    if (top == -INFINITY) top = 0.0;  // no expert can be chosen
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      c[i] = exp((double)x[i] - top);
      part += c[i];
    }
    sum = wave_sum_f64(part);
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    const float b = bias && e < p.E ? bias[e] : 0.0f;
    const double s = p.sigmoid ? sigmoid_scaled(x[i], 0.0) : (sum > 0.0 || isnan(sum) ? c[i] / sum : 0.0);
    bad |= isnan(x[i]) || isnan(b) || isnan(s);
    c[i] = x[i] == -INFINITY || b == -INFINITY ? -INFINITY : s + b;
  }
  if (__ballot(bad)) {
    if (lane < p.k) {
      ids[lane] = -1;
      w[lane] = NAN;
    }
    return;
  }
  if (p.groups > 1) {
    const int each = p.E / p.groups;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sh[lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    double b1 = -INFINITY, b2 = -INFINITY;
    if (lane < p.groups)
      for (int i = 0; i < each; ++i) {
        const double v = sh[lane * each + i];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
    const double v = p.group_best == 2 && b2 > -INFINITY ? b1 + b2 : b1;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const double o = __shfl(v, g, 64);
      rank += o > v || (o == v && g < lane);
    }
    const uint64_t stay = __ballot(lane < p.groups && rank < p.group_topk && v > -INFINITY);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e >= p.E || !((stay >> (e / each)) & 1)) c[i] = -INFINITY;
    }
  }
  int mine = -1;
  for (int j = 0; j < p.k; ++j) {
    double bv = -INFINITY;
    int be = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (c[i] > bv) {  // ids rise with i: a tie keeps the lower one
        bv = c[i];
        be = lane + 64 * i;
      }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
      const double ov = __shfl_xor(bv, m, 64);
      const int oe = __shfl_xor(be, m, 64);
      if (ov > bv || (ov == bv && oe < be)) {
        bv = ov;
        be = oe;
      }
    }
    if (be == 0x7FFFFFFF) break;  // the same in every lane
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (be == lane + 64 * i) c[i] = -INFINITY;
    if (lane == j) mine = be;
  }
  const bool there = mine >= 0;
  const double q = chosen_weight(p, there, there ? (double)row[mine] : 0.0, top, sum);
  if (lane < p.k) {
    ids[lane] = mine;
    w[lane] = (float)(q * p.scale);
  }
}

template <int EPL>
__global__ __launch_bounds__(256) void score_choose_kernel(const ScoreArgs p, const float* __restrict__ logits,
                                                           const float* __restrict__ bias,
                                                           const uint8_t* __restrict__ mask, int32_t* __restrict__ ids,
                                                           float* __restrict__ w) {
  __shared__ double sh_c[4][EPL * 64];
  const int wv = threadIdx.x >> 6;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wv; t < p.T; t += (int64_t)gridDim.x * 4)
    score_choose_token<EPL>(p, logits + t * p.E, bias, mask && mask[t] == 0, sh_c[wv], ids + t * p.k, w + t * p.k);
}

size_t score_ws_bytes(int64_t T, int64_t E, int64_t k) { return plan_ws_bytes(T * k, E); }

hipError_t launch_score_route(const ScoreArgs& p, const float* logits, const float* bias, const uint8_t* mask,
                              int32_t* ids, float* w, int32_t* counts, int32_t* offsets, int32_t* perm,
                              int32_t* inv_perm, void* ws, hipStream_t st) {
  if (p.T > 0) {
    const dim3 grid(token_grid(p.T)), block(256);
    if (p.E <= 64) score_choose_kernel<1><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    else if (p.E <= 128) score_choose_kernel<2><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    else if (p.E <= 256) score_choose_kernel<4><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    else if (p.E <= 512) score_choose_kernel<8><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    else score_choose_kernel<16><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_plan(ids, (int64_t)p.T * p.k, p.E, counts, offsets, perm, inv_perm, ws, st);
}

// -------------------------------------------------------------------------------- backward
// One wave per token; lane j < k holds slot j, and the lanes then write the row.
template <int EPL>
__device__ __forceinline__ void score_backward_token(const ScoreArgs& p, const float* __restrict__ row,
                                                     const int32_t* __restrict__ ids, const float* __restrict__ d_w,
                                                     float* __restrict__ d) {
  const int lane = threadIdx.x & 63;
  const int id = lane < p.k ? ids[lane] : -1;
  const bool there = id >= 0 && id < p.E;
  const double g = there ? (double)d_w[lane] * p.scale : 0.0;
  const double l = there ? (double)row[id] : 0.0;
  const bool any = __ballot(there) != 0;
  const bool dense = any && !p.sigmoid && !p.renorm;
  float x[EPL], out[EPL];
  double top = 0.0, sum = 1.0;
  if (dense) {
    float xmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      x[i] = e < p.E ? row[e] : -INFINITY;
      xmax = fmaxf(xmax, x[i]);
    }
    top = wave_max_f64(xmax);
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) part += x[i] = expf(x[i] - (float)top);
    sum = wave_sum_f64(part);
  }
  const double q = chosen_weight(p, there, l, top, sum);
  const double dot = p.renorm || dense ? wave_sum_f64(g * q) : 0.0;
  // what slot j adds at its expert
  float v = 0.0f;
  if (there) v = (float)(dense ? g : p.sigmoid ? (g - dot) * q * sigmoid_scaled(-l, 0.0) : (g - dot) * q);
#pragma unroll
  for (int i = 0; i < EPL; ++i) out[i] = dense ? -(float)dot : 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const int e = __shfl(id, j, 64);
    const float u = __shfl(v, j, 64);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e == lane + 64 * i) out[i] += u;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e < p.E) d[e] = dense ? out[i] * (x[i] / (float)sum) : out[i];
  }
}

template <int EPL>
__global__ __launch_bounds__(256) void score_backward_kernel(const ScoreArgs p, const float* __restrict__ logits,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ d_w, float* __restrict__ d) {
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < p.T; t += (int64_t)gridDim.x * 4)
    score_backward_token<EPL>(p, logits + t * p.E, ids + t * p.k, d_w + t * p.k, d + t * p.E);
}

hipError_t launch_score_backward(const ScoreArgs& p, const float* logits, const int32_t* ids, const float* d_w,
                                 float* d_logits, hipStream_t st) {
  const dim3 grid(token_grid(p.T)), block(256);
  if (p.E <= 64) score_backward_kernel<1><<<grid, block, 0, st>>>(p, logits, ids, d_w, d_logits);
  else if (p.E <= 128) score_backward_kernel<2><<<grid, block, 0, st>>>(p, logits, ids, d_w, d_logits);
  else if (p.E <= 256) score_backward_kernel<4><<<grid, block, 0, st>>>(p, logits, ids, d_w, d_logits);
  else if (p.E <= 512) score_backward_kernel<8><<<grid, block, 0, st>>>(p, logits, ids, d_w, d_logits);
  else score_backward_kernel<16><<<grid, block, 0, st>>>(p, logits, ids, d_w, d_logits);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------ bias
// One block: the counts' sum in whole numbers, then each bias one step towards an even load.
__global__ __launch_bounds__(1024) void bias_update_kernel(int E, const int32_t* __restrict__ counts, float rate,
                                                           const float* bias, float* out) {
  __shared__ int64_t part[16];
  const int e = threadIdx.x, lane = e & 63;
  const int64_t n = e < E ? counts[e] : 0;
  int64_t sum = n;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m, 64);
  if (lane == 0) part[e >> 6] = sum;
  __syncthreads();
  if (e >= E) return;
  int64_t total = 0;
  for (int i = 0; i < (int)blockDim.x / 64; ++i) total += part[i];
  const int64_t over = n * E - total;
  out[e] = bias[e] + (over > 0 ? -rate : over < 0 ? rate : 0.0f);
}

hipError_t launch_bias_update(int E, const int32_t* counts, float rate, const float* bias, float* out, hipStream_t st) {
  bias_update_kernel<<<1, (E + 63) / 64 * 64, 0, st>>>(E, counts, rate, bias, out);
  return hipGetLastError();
}

}  // namespace moe
