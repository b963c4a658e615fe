// Gradient norm and AdamW step over a list of tensors.
//
//   norm = sqrt(sum g^2),  scale = min(1, max_norm / (norm + 1e-6))
//   g' = scale g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   w = (1 - lr wd) w - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
// The weights' master copies stay in more bits than the layer computes with (page "NVIDIA מציגה
// דרך יעילה לאמן מודלי MoE בביולוגיה", section "צמצום הזיכרון ותקורות הכימות").
//
// 8-bit states hold m and sqrt(v) as e4m3 codes with one fp32 scale (largest magnitude / 448) for
// each 256 values.  They are rounded stochastically: an average moves by (1 - b) of its distance
// in a step, far less than half of e4m3's step of 1/8, so rounding to nearest would hold it where
// it is; rounded up with the probability of the remainder its expectation moves as it should.
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kChunk = 4096;  // values a block updates: 4 waves x 4 runs of 256

enum { kAdamP32 = 1, kAdamG32 = 2, kAdam8bit = 4 };

struct AdamTensor {
  void* p;
  const void* g;
  void *m, *v;
  float *m_scale, *v_scale, *master;
  int64_t n;
  float weight_decay;
  int32_t flags;
};

struct AdamBatch {
  AdamTensor t[kAdamBatch];
  int32_t first[kAdamBatch + 1];  // first chunk of each tensor
  int32_t n;
};
static_assert(sizeof(AdamBatch) + sizeof(AdamScalars) <= 4096 - 64, "kernel arguments");

__device__ __forceinline__ int tensor_of(const AdamBatch& b, int chunk) {
  int lo = 0, hi = b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// 1 - beta^step by squaring, in 64 bits
__device__ __forceinline__ double one_less_power(double beta, uint64_t step) {
  double p = 1.0, q = beta;
  for (; step; step >>= 1, q *= q)
    if (step & 1) p *= q;
  return 1.0 - p;
}

// Random words of the element: the step's keys are splitmix64's finaliser (Steele, Lea, Flood 2014)
// of the seed, the step and the tensor's place in the list; each value's words come from them and
// its index by two and three rounds of multiply and shift (the constants: of 400 random odd pairs
// the one whose words of neighbouring values are least alike; they are as independent as chance).
__device__ __forceinline__ uint64_t step_key(uint64_t seed, uint64_t step, uint64_t tensor) {
  uint64_t z = (seed ^ (step << 32) ^ tensor) + 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

__device__ __forceinline__ uint32_t noise(uint32_t k0, uint32_t k1, int64_t i) {
  uint32_t u = ((uint32_t)i + (uint32_t)(i >> 32) * 0x9E3779B9u) ^ k0;
  u = (u ^ (u >> 16)) * 0x32A0CD0Bu;
  u = (u ^ (u >> 14) ^ k1) * 0x2F37D463u;
  return u ^ (u >> 16);
}

__device__ __forceinline__ uint32_t noise2(uint32_t u, uint32_t k0) {
  const uint32_t w = (u ^ k0) * 0xBB67AE85u;
  return w ^ (w >> 15);
}

// e4m3 code of y in [0, 448], rounded up with the probability of the remainder (16 random bits).
// Below 2^-6 the codes are even steps of 2^-9: 2^-6 added makes them those of one binade.
__device__ __forceinline__ uint32_t code_of(float y, uint32_t r16) {
  const bool low = y < 0.015625f;
  const uint32_t b = __float_as_uint(low ? y + 0.015625f : y) + (r16 << 4);
  return (b >> 20) - (low ? 968u : 960u);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
  return v;
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));

// 4 consecutive values from element i; with `ok` < 4 only the first ones exist
__device__ __forceinline__ void load4(const void* p, int64_t i, int ok, bool f32, float (&x)[4]) {
  if (ok == 4) {
    if (f32) {
      const float4 q = *(const float4*)((const float*)p + i);
      x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
    } else {
      const uint2 q = *(const uint2*)((const uint16_t*)p + i);
      x[0] = lo_bf16(q.x), x[1] = hi_bf16(q.x), x[2] = lo_bf16(q.y), x[3] = hi_bf16(q.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[j] = j < ok ? (f32 ? ((const float*)p)[i + j] : bf16_to_f32(((const uint16_t*)p)[i + j])) : 0.0f;
  }
}

__device__ __forceinline__ void store4f(float* p, int64_t i, int ok, const float (&x)[4]) {
  if (ok == 4) {
    *(float4*)(p + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < ok) p[i + j] = x[j];
  }
}

__device__ __forceinline__ void store4h(uint16_t* p, int64_t i, int ok, uint32_t a, uint32_t b) {
  if (ok == 4) {
    *(uint2*)(p + i) = make_uint2(a, b);
  } else {
    const uint32_t w[2] = {a, b};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < ok) p[i + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}

__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t i, int ok) {
  if (ok == 4) return *(const uint32_t*)(p + i);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < ok) w |= (uint32_t)p[i + j] << (8 * j);
  return w;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int ok, uint32_t w) {
  if (ok == 4) {
    *(uint32_t*)(p + i) = w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < ok) p[i + j] = (uint8_t)(w >> (8 * j));
  }
}

__device__ __forceinline__ void decode4(uint32_t w, float scale, float (&x)[4]) {
  const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  x[0] = a[0] * scale, x[1] = a[1] * scale, x[2] = b[0] * scale, x[3] = b[1] * scale;
}

// scale of a block with largest magnitude `top`: top / 448 by a product, within one unit of it
__device__ __forceinline__ float block_scale(float top) {
  return top > 0.0f ? fmaxf(top * (1.0f / 448.0f), 1.17549435e-38f) : 1.0f;
}

// Products and sums round one by one (no fused multiply-add): a state's code then follows from
// single fp32 operations, and the same step written out in them gives the same bits.
__global__ __launch_bounds__(256) void adamw_kernel(AdamBatch batch, AdamScalars hp) {
#pragma clang fp contract(off)
  float gs = 1.0f;
  if (hp.d_grad_scale) {
    gs = *hp.d_grad_scale;
    if (!(fabsf(gs) < INFINITY)) return;  // a step to skip: nothing changes
  }
  const int which = tensor_of(batch, blockIdx.x);
  const AdamTensor& T = batch.t[which];
  const float lr = hp.d_lr ? *hp.d_lr : hp.lr;
  float inv_c1 = hp.inv_c1, inv_rc2 = hp.inv_rc2;
  uint64_t step = hp.step;
  if (hp.d_step) {
    step = (uint64_t)*hp.d_step;
    inv_c1 = (float)(1.0 / one_less_power(hp.b1d, step));
    inv_rc2 = (float)(1.0 / sqrt(one_less_power(hp.b2d, step)));
  }
  const uint64_t key = step_key(hp.seed, step, (uint64_t)(hp.first_tensor + which));
  const uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
  const float keep = 1.0f - lr * T.weight_decay, rate = lr * inv_c1;
  const bool p32 = T.flags & kAdamP32, g32 = T.flags & kAdamG32, eight = T.flags & kAdam8bit;
  const bool random_p = !p32 && !T.master && hp.stochastic;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t base = (int64_t)(blockIdx.x - batch.first[which]) * kChunk;
#pragma unroll 2
  for (int it = 0; it < kChunk / 1024; ++it) {
    const int64_t i0 = base + (it * 4 + wv) * 256, i = i0 + lane * 4;
    if (i0 >= T.n) return;
    const int64_t left = T.n - i;
    const int ok = left >= 4 ? 4 : left > 0 ? (int)left : 0;
    float g[4], m[4], v[4], w[4], root[4];
    load4(T.g, i, ok, g32, g);
    if (T.master) load4(T.master, i, ok, true, w);
    else load4(T.p, i, ok, p32, w);
    if (eight) {
      decode4(load_codes((const uint8_t*)T.m, i, ok), T.m_scale[i0 / 256], m);
      decode4(load_codes((const uint8_t*)T.v, i, ok), T.v_scale[i0 / 256], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= v[j];
    } else {
      load4(T.m, i, ok, true, m);
      load4(T.v, i, ok, true, v);
    }
    uint32_t u[4] = {0, 0, 0, 0};
    if (eight || random_p)
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = noise(k0, k1, i + j);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g[j] *= gs;
      m[j] = hp.b1 * m[j] + hp.a1 * g[j];
      v[j] = hp.b2 * v[j] + (hp.a2 * g[j]) * g[j];
      root[j] = sqrtf(v[j]);
      w[j] = w[j] * keep - rate * m[j] / (root[j] * inv_rc2 + hp.eps);
    }
    if (T.master) store4f(T.master, i, ok, w);
    if (p32) {
      store4f((float*)T.p, i, ok, w);
    } else if (random_p) {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = (__float_as_uint(w[j]) + (noise2(u[j], k0) & 0xFFFFu)) >> 16;
      store4h((uint16_t*)T.p, i, ok, b[0] | b[1] << 16, b[2] | b[3] << 16);
    } else {
      store4h((uint16_t*)T.p, i, ok, pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]));
    }
    if (eight) {
      float tm = 0.0f, tr = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < ok) tm = fmaxf(tm, fabsf(m[j])), tr = fmaxf(tr, root[j]);
      const float sm = block_scale(wave_max(tm)), sr = block_scale(wave_max(tr));
      const float im = 1.0f / sm, ir = 1.0f / sr;
      uint32_t cm = 0, cr = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = code_of(fminf(fabsf(m[j]) * im, 448.0f), u[j] & 0xFFFFu);
        cm |= (a | (m[j] < 0.0f ? 0x80u : 0u)) << (8 * j);
        const float y = fminf(root[j] * ir, 448.0f);
        uint32_t b = code_of(y, u[j] >> 16);
        if (b == 0 && y > 0.0f) b = 1;  // a root above 0 stays above 0: it divides the next step
        cr |= b << (8 * j);
      }
      store_codes((uint8_t*)T.m, i, ok, cm);
      store_codes((uint8_t*)T.v, i, ok, cr);
      if (lane == 0) T.m_scale[i0 / 256] = sm, T.v_scale[i0 / 256] = sr;
    } else {
      store4f((float*)T.m, i, ok, m);
      store4f((float*)T.v, i, ok, v);
    }
  }
}

// Sum of g^2 of one chunk, in 64 bits (no square of an fp32 value overflows or vanishes there).
__global__ __launch_bounds__(256) void grad_norm_kernel(AdamBatch batch, int chunk, double* __restrict__ part) {
  __shared__ double sh[4];
  const int which = tensor_of(batch, blockIdx.x);
  const AdamTensor& T = batch.t[which];
  const bool g32 = T.flags & kAdamG32;
  const int64_t a = (int64_t)(blockIdx.x - batch.first[which]) * chunk;
  const int64_t z = T.n - a < chunk ? T.n : a + chunk;
  double s = 0.0;
#pragma unroll 4
  for (int64_t i = a + threadIdx.x * 4; i < z; i += 1024) {
    const int64_t left = z - i;
    float g[4];
    load4(T.g, i, left >= 4 ? 4 : (int)left, g32, g);
#pragma unroll
    for (int j = 0; j < 4; ++j) s += (double)g[j] * (double)g[j];
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

__global__ __launch_bounds__(1024) void grad_norm_final_kernel(const double* __restrict__ part, int64_t n, float max_norm,
                                                               float* __restrict__ norm, float* __restrict__ scale) {
  __shared__ double sh[16];
  double s = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += part[i];
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = 0.0;
  for (int w = 0; w < 16; ++w) s += sh[w];
  const double r = sqrt(s);
  *norm = (float)r;
  if (scale) {
    const double f = (double)max_norm / (r + 1e-6);
    *scale = !((float)r < INFINITY) ? NAN : f < 1.0 ? (float)f : 1.0f;  // NaN: a step to skip
  }
}

// Calls fn(batch, chunks, index of the batch's first tensor) for runs of up to kAdamBatch tensors
// that are not empty, each cut into chunks of `chunk` values.
template <class F>
hipError_t for_batches(const moe_tensor* t, int64_t n, int64_t chunk, F fn) {
  AdamBatch b;
  b.n = 0;
  int64_t chunks = 0, first = 0;
  for (int64_t i = 0; i < n; ++i) {
    const int64_t c = (t[i].n + chunk - 1) / chunk;
    if (b.n == kAdamBatch || (b.n > 0 && chunks + c >= ((int64_t)1 << 31))) {
      b.first[b.n] = (int32_t)chunks;
      const hipError_t e = fn(b, chunks, first);
      if (e != hipSuccess) return e;
      b.n = 0;
      chunks = 0;
    }
    if (b.n == 0) first = i;
    b.t[b.n] = AdamTensor{t[i].p, t[i].g, t[i].m, t[i].v, t[i].m_scale, t[i].v_scale, t[i].master, t[i].n,
                          t[i].weight_decay,
                          (t[i].p_dtype == MOE_F32 ? kAdamP32 : 0) | (t[i].g_dtype == MOE_F32 ? kAdamG32 : 0) |
                              (t[i].state == MOE_STATE_8BIT ? kAdam8bit : 0)};
    b.first[b.n++] = (int32_t)chunks;
    chunks += c;
  }
  if (b.n == 0 || chunks == 0) return hipSuccess;
  b.first[b.n] = (int32_t)chunks;
  return fn(b, chunks, first);
}

int64_t norm_chunk(const moe_tensor* t, int64_t n) {
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) total += t[i].n;
  const int64_t c = (total / 4096 + 4095) / 4096 * 4096;  // about 4096 blocks
  return c < 4096 ? 4096 : c > ((int64_t)1 << 30) ? (int64_t)1 << 30 : c;
}

int64_t norm_chunks(const moe_tensor* t, int64_t n, int64_t chunk) {
  int64_t k = 0;
  for (int64_t i = 0; i < n; ++i) k += (t[i].n + chunk - 1) / chunk;
  return k;
}

}  // namespace

hipError_t launch_adamw(const moe_tensor* t, int64_t n, const AdamScalars& hp, hipStream_t st) {
  return for_batches(t, n, kChunk, [&](const AdamBatch& b, int64_t chunks, int64_t first) {
    AdamScalars h = hp;
    h.first_tensor = first;
    adamw_kernel<<<(unsigned)chunks, 256, 0, st>>>(b, h);
    return hipGetLastError();
  });
}

size_t grad_norm_ws_bytes(const moe_tensor* t, int64_t n) { return (size_t)norm_chunks(t, n, norm_chunk(t, n)) * 8; }

hipError_t launch_grad_norm(const moe_tensor* t, int64_t n, float max_norm, float* norm, float* scale, double* part,
                            hipStream_t st) {
  const int64_t chunk = norm_chunk(t, n);
  int64_t at = 0;
  const hipError_t e = for_batches(t, n, chunk, [&](const AdamBatch& b, int64_t chunks, int64_t) {
    grad_norm_kernel<<<(unsigned)chunks, 256, 0, st>>>(b, (int)chunk, part + at);
    at += chunks;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  grad_norm_final_kernel<<<1, 1024, 0, st>>>(part, at, max_norm, norm, scale);
  return hipGetLastError();
}

}  // namespace moe
