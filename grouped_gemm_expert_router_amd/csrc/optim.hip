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
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// A block of the update: a wave takes 256 values.  fp32 states move 22 to 30 bytes a value in seven or eight
// streams, and DRAM serves them best from few waves in small blocks: with one wave a block and three a SIMD,
// 604M weights with master copies take 2.62 ms; four a SIMD 2.65, eight in blocks of four 3.02 (bf16
// weights without master copies: 200M in 0.81 ms, 0.76, 0.84).  8-bit states are nearer the vector ALU's
// bound and want every wave: 1.55 ms, one wave a block 1.6, five a SIMD 1.69.
constexpr int adam_threads(bool eight) { return eight ? 256 : 64; }
constexpr int adam_chunk(bool eight) { return adam_threads(eight) * 4; }

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

// Tensors of one launch, in its arguments; first: first chunk of each, modulo 2^32 (the first tensor's
// lies before the launch if earlier ones took some of it).  Lists without 8-bit states leave the scales out and fit more tensors in a launch (60 tensors of
// 3333 values: 6.6 us, in two launches 10.0).
template <bool EIGHT>
struct AdamBatch {
  static constexpr bool kEight = EIGHT;
  static constexpr int kMost = EIGHT ? 54 : 64;
  void* ptr[EIGHT ? 7 : 5][kMost];  // p, g, m, v, master, scales
  int64_t n8[kMost];                // 8 n + flags
  float weight_decay[kMost];
  int32_t first[kMost];
  int32_t n;
  void put(const moe_tensor& q) {
    ptr[0][n] = q.p, ptr[1][n] = (void*)q.g, ptr[2][n] = q.m, ptr[3][n] = q.v, ptr[4][n] = q.master;
    if constexpr (EIGHT) ptr[5][n] = q.m_scale, ptr[6][n] = q.v_scale;
    n8[n] = 8 * q.n + (q.p_dtype == MOE_F32 ? kAdamP32 : 0) + (q.g_dtype == MOE_F32 ? kAdamG32 : 0) +
            (q.state == MOE_STATE_8BIT ? kAdam8bit : 0);
    weight_decay[n] = q.weight_decay;
  }
  __device__ __forceinline__ AdamTensor get(int i) const {
    AdamTensor t{ptr[0][i], ptr[1][i], ptr[2][i], ptr[3][i], nullptr, nullptr, (float*)ptr[4][i],
                 n8[i] >> 3, weight_decay[i], (int32_t)(n8[i] & 7)};
    if constexpr (EIGHT) t.m_scale = (float*)ptr[5][i], t.v_scale = (float*)ptr[6][i];
    return t;
  }
};
static_assert(sizeof(AdamBatch<false>) + sizeof(AdamScalars) <= 4096 - 64, "kernel arguments");
static_assert(sizeof(AdamBatch<true>) + sizeof(AdamScalars) <= 4096 - 64, "kernel arguments");

struct GradBatch {
  static constexpr int kMost = 3 * 64;
  const void* g[kMost];
  int64_t n32[kMost];  // 2 n + 1 for fp32 gradients, 2 n for bf16
  int32_t first[kMost];
  int32_t n;
  void put(const moe_tensor& q) {
    g[n] = q.g;
    n32[n] = 2 * q.n + (q.g_dtype == MOE_F32);
  }
};
static_assert(sizeof(GradBatch) <= 4096 - 64, "kernel arguments");

// The tensor of a chunk: each lane compares an entry or a few (the arguments may lie in host memory,
// where a search's dependent reads cost a round trip each).
template <class Batch>
__device__ __forceinline__ int tensor_of(const Batch& b, int chunk) {
  int at = -1;
#pragma unroll
  for (int q = 0; q < Batch::kMost; q += 64) {
    const int i = q + (threadIdx.x & 63);
    at += __popcll(__ballot(i < b.n && (i == 0 || b.first[i < Batch::kMost ? i : 0] <= chunk)));
  }
  return at;
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

// e4m3 code of y in [0, 448], rounded up with the probability of the remainder: rs holds 16 random bits
// in place (bits 4 to 19 of the 20 that the code leaves out).  A code is an fp32 value's exponent less
// 120 and its upper three mantissa bits; below 2^-6 the codes are even steps of 2^-9, those of one
// binade once 2^-6 is added, and half of that has the exponent one lower that they start from.
__device__ __forceinline__ uint32_t code_of(float y, uint32_t rs) {
  const uint32_t b = __float_as_uint(y < 0.015625f ? __builtin_fmaf(y, 0.5f, 0.0078125f) : y);
  return (b + rs - (960u << 20)) >> 20;
}

// Square root: the hardware's reciprocal root (1 ulp) and one correction of the product.  The same bits
// as the rounded root for every mantissa in two binades, normal and denormal (checked on the GPU); 0 and
// infinity are their own roots.
__device__ __forceinline__ float root_of(float v) {
  const bool tiny = v < 0x1p-96f;  // keeps the reciprocal's argument normal
  const float x = tiny ? v * 0x1p64f : v;
  const float y = __builtin_amdgcn_rsqf(x), r = x * y;
  float q = __builtin_fmaf(__builtin_fmaf(-r, r, x), 0.5f * y, r);
  if (tiny) q *= 0x1p-32f;
  return __builtin_amdgcn_classf(v, 0x260) ? v : q;
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// 4 consecutive values from element i
template <bool F32>
__device__ __forceinline__ void load4(const void* p, int64_t i, float (&x)[4]) {
  if (F32) {
    const f32x4_t q = __builtin_nontemporal_load((const f32x4_t*)((const float*)p + i));
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = q[j];
  } else {
    const u32x2_t q = __builtin_nontemporal_load((const u32x2_t*)((const uint16_t*)p + i));
    x[0] = lo_bf16(q[0]), x[1] = hi_bf16(q[0]), x[2] = lo_bf16(q[1]), x[3] = hi_bf16(q[1]);
  }
}

__device__ __forceinline__ void store4(void* p, int64_t i, const float (&x)[4]) {
  __builtin_nontemporal_store(f32x4_t{x[0], x[1], x[2], x[3]}, (f32x4_t*)((float*)p + i));
}

__device__ __forceinline__ void store4(void* p, int64_t i, uint32_t a, uint32_t b) {
  __builtin_nontemporal_store(u32x2_t{a, b}, (u32x2_t*)((uint16_t*)p + i));
}

__device__ __forceinline__ void decode4(uint32_t w, float scale, float (&x)[4]) {
  const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  x[0] = a[0] * scale, x[1] = a[1] * scale, x[2] = b[0] * scale, x[3] = b[1] * scale;
}

// scale of a block with largest magnitude `top`: top / 448 by a product, within one unit of it
__device__ __forceinline__ float block_scale(float top) {
  return top > 0.0f ? fmaxf(top * (1.0f / 448.0f), 1.17549435e-38f) : 1.0f;
}

// 1 / s for a normal s: the hardware's reciprocal (1 ulp) and one Newton step
__device__ __forceinline__ float inverse(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return __fmaf_rn(__fmaf_rn(-s, r, 1.0f), r, r);
}

// What a step needs beside the tensors, the same for a whole launch or tensor
struct Step {
  float b1, b2, a1, a2, eps, gs, keep, rate, inv_rc2;
  uint32_t k0, k1;
  bool random_p;
};

// Four values' update; `w` holds the master copy or the parameter.  The moments' products and sums
// round one by one (no fused multiply-add): a state's code then follows from single fp32 operations,
// and the same step written out in them gives the same bits.
__device__ __forceinline__ void update4(const Step& h, float (&g)[4], float (&m)[4], float (&v)[4], float (&w)[4],
                                        float (&root)[4]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    g[j] *= h.gs;
    m[j] = h.b1 * m[j] + h.a1 * g[j];
    v[j] = h.b2 * v[j] + (h.a2 * g[j]) * g[j];
    root[j] = root_of(v[j]);
    w[j] = __builtin_fmaf(w[j], h.keep, -(h.rate * m[j]) * __builtin_amdgcn_rcpf(__builtin_fmaf(root[j], h.inv_rc2, h.eps)));
  }
}

// Four values' codes of m and sqrt(v) and their 256 values' scales (a whole wave calls it).
__device__ __forceinline__ void encode4(const float (&m)[4], const float (&root)[4], const uint32_t (&u)[4],
                                        uint32_t& cm, uint32_t& cr, float& sm, float& sr) {
#pragma clang fp contract(off)
  sm = block_scale(wave_max_dpp(fmaxf(fmaxf(fabsf(m[0]), fabsf(m[1])), fmaxf(fabsf(m[2]), fabsf(m[3])))));
  sr = block_scale(wave_max_dpp(fmaxf(fmaxf(root[0], root[1]), fmaxf(root[2], root[3]))));
  const float im = inverse(sm), ir = inverse(sr);
  cm = cr = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = code_of(fminf(fabsf(m[j]) * im, 448.0f), (u[j] << 4) & 0xFFFF0u);
    cm |= (a | (__float_as_uint(m[j]) >> 24 & 0x80u)) << (8 * j);
    const float y = fminf(root[j] * ir, 448.0f);
    // a root above 0 stays above 0: it divides the next step
    const uint32_t least = __float_as_uint(y) < 1u ? 0u : 1u, b = code_of(y, (u[j] >> 12) & 0xFFFF0u);
    cr |= (b > least ? b : least) << (8 * j);
  }
}

// Two bf16 pairs of w, stochastically rounded with the second words of u (a NaN's bits could carry into
// its sign)
__device__ __forceinline__ void random4(const float (&w)[4], const uint32_t (&u)[4], uint32_t k0, uint32_t& a, uint32_t& b) {
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    q[j] = w[j] == w[j] ? (__float_as_uint(w[j]) + (noise2(u[j], k0) & 0xFFFFu)) >> 16 : 0x7FC0u;
  a = q[0] | q[1] << 16;
  b = q[2] | q[3] << 16;
}

// The 256 whole values of a wave from b: every load is issued before the first use.  The streams are
// read and written once (non-temporal).  Bound by HBM: 604M bf16 weights with fp32 master copies take
// 2.62 ms with fp32 states (28 bytes a value, 6.5 TB/s) and 1.55 ms with 8-bit states (16, 6.2 TB/s).
// One run a wave and no more (in blocks of four waves, as many as fit: 2.95 and 1.60 ms; 4 runs of a wave in
// turn 3.08 and 1.72, two of them in flight together 3.02 and 1.66; cached stores 3.11 and 1.79).  The
// step's number on the device costs a wave an expm1: 8-bit states 1.73 ms (by powers in 64 bits in every
// lane: 2.15 to 2.39).  200M weights without master copies: fp32 0.89 ms (6.3 TB/s) and with 8-bit states
// 0.53 (6.1); bf16, rounded with random bits, 0.81 (5.4) and with 8-bit states 0.49 (4.1: nearer the vector
// ALU's bound, two random words a value).
template <bool P32, bool MASTER, bool G32, bool EIGHT>
__device__ __forceinline__ void adamw_run(const AdamTensor& T, const Step& h, int64_t b, int lane) {
  const int64_t i = b + lane * 4;
  float g[4], m[4], v[4], w[4], root[4];
  uint32_t qm, qv, u[4];
  float sm, sv;
  load4<G32>(T.g, i, g);
  if (MASTER) load4<true>(T.master, i, w);
  else load4<P32>(T.p, i, w);
  if (EIGHT) {
    qm = __builtin_nontemporal_load((const uint32_t*)((const uint8_t*)T.m + i));
    qv = __builtin_nontemporal_load((const uint32_t*)((const uint8_t*)T.v + i));
    sm = T.m_scale[b / 256];
    sv = T.v_scale[b / 256];
    decode4(qm, sm, m);
    decode4(qv, sv, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= v[j];
  } else {
    load4<true>(T.m, i, m);
    load4<true>(T.v, i, v);
  }
  if (EIGHT || (!P32 && !MASTER))
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = noise(h.k0, h.k1, i + j);
  update4(h, g, m, v, w, root);
  if (MASTER) store4(T.master, i, w);
  if (P32) {
    store4(T.p, i, w);
  } else if (!MASTER && h.random_p) {
    uint32_t x, y;
    random4(w, u, h.k0, x, y);
    store4(T.p, i, x, y);
  } else {
    store4(T.p, i, pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]));
  }
  if (EIGHT) {
    encode4(m, root, u, qm, qv, sm, sv);
    __builtin_nontemporal_store(qm, (uint32_t*)((uint8_t*)T.m + i));
    __builtin_nontemporal_store(qv, (uint32_t*)((uint8_t*)T.v + i));
    if (lane == 0) T.m_scale[b / 256] = sm, T.v_scale[b / 256] = sv;
  } else {
    store4(T.m, i, m);
    store4(T.v, i, v);
  }
}

// The last run of a tensor, shorter than 256: value by value.
template <bool EIGHT>
__device__ __forceinline__ void adamw_tail(const AdamTensor& T, const Step& h, int64_t i0, int lane) {
  const bool p32 = T.flags & kAdamP32, g32 = T.flags & kAdamG32, eight = EIGHT && T.flags & kAdam8bit;
  const int64_t i = i0 + lane * 4;
  float g[4], m[4], v[4], w[4], root[4];
  uint32_t u[4], cm = 0, cr = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    g[j] = m[j] = v[j] = w[j] = 0.0f;
    u[j] = noise(h.k0, h.k1, i + j);
    if (i + j >= T.n) continue;
    g[j] = g32 ? ((const float*)T.g)[i + j] : bf16_to_f32(((const uint16_t*)T.g)[i + j]);
    w[j] = T.master ? T.master[i + j] : p32 ? ((const float*)T.p)[i + j] : bf16_to_f32(((const uint16_t*)T.p)[i + j]);
    if (eight) {
      cm |= (uint32_t)((const uint8_t*)T.m)[i + j] << (8 * j);
      cr |= (uint32_t)((const uint8_t*)T.v)[i + j] << (8 * j);
    } else {
      m[j] = ((const float*)T.m)[i + j];
      v[j] = ((const float*)T.v)[i + j];
    }
  }
  if (eight) {
    decode4(cm, T.m_scale[i0 / 256], m);
    decode4(cr, T.v_scale[i0 / 256], v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= v[j];
  }
  update4(h, g, m, v, w, root);  // 0 stays 0 behind the last value
  uint32_t b[2] = {pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3])};
  if (h.random_p) random4(w, u, h.k0, b[0], b[1]);
  float sm = 0.0f, sr = 0.0f;
  if (eight) {
    encode4(m, root, u, cm, cr, sm, sr);
    if (lane == 0) T.m_scale[i0 / 256] = sm, T.v_scale[i0 / 256] = sr;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (i + j >= T.n) continue;
    if (T.master) T.master[i + j] = w[j];
    if (p32) ((float*)T.p)[i + j] = w[j];
    else ((uint16_t*)T.p)[i + j] = (uint16_t)(b[j >> 1] >> (16 * (j & 1)));
    if (eight) {
      ((uint8_t*)T.m)[i + j] = (uint8_t)(cm >> (8 * j));
      ((uint8_t*)T.v)[i + j] = (uint8_t)(cr >> (8 * j));
    } else {
      ((float*)T.m)[i + j] = m[j];
      ((float*)T.v)[i + j] = v[j];
    }
  }
}

}  // namespace

template <bool EIGHT>
__global__ __launch_bounds__(adam_threads(EIGHT)) __attribute__((amdgpu_waves_per_eu(EIGHT ? 1 : 3, EIGHT ? 8 : 3)))
void adamw_kernel(AdamBatch<EIGHT> batch, AdamScalars hp) {
  Step h;
  h.gs = 1.0f;
  if (hp.d_grad_scale) {
    h.gs = *hp.d_grad_scale;
    if (!(fabsf(h.gs) < INFINITY)) return;  // a step to skip: nothing changes
  }
  const int which = tensor_of(batch, blockIdx.x);
  const AdamTensor T = batch.get(which);
  const float lr = hp.d_lr ? *hp.d_lr : hp.lr;
  float inv_c1 = hp.inv_c1;
  h.inv_rc2 = hp.inv_rc2;
  uint64_t step = hp.step;
  if (hp.d_step) {
    // 1 - beta^step = -expm1(step ln beta): beta1 in the even lanes, beta2 in the odd ones
    step = (uint64_t)*hp.d_step;
    const float c = -expm1f((float)((double)step * (threadIdx.x & 1 ? hp.ln_b2 : hp.ln_b1)));
    const float inv = inverse(c);
    inv_c1 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv), 0));
    h.inv_rc2 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(__builtin_amdgcn_sqrtf(inv)), 1));
  }
  const uint64_t key = step_key(hp.seed, step, (uint64_t)(hp.first_tensor + which));
  h.k0 = (uint32_t)key, h.k1 = (uint32_t)(key >> 32);
  h.b1 = hp.b1, h.b2 = hp.b2, h.a1 = hp.a1, h.a2 = hp.a2, h.eps = hp.eps;
  h.keep = 1.0f - lr * T.weight_decay;
  h.rate = lr * inv_c1;
  h.random_p = !(T.flags & kAdamP32) && !T.master && hp.stochastic;
  const int lane = threadIdx.x & 63;
  const int64_t b = (int64_t)(blockIdx.x - batch.first[which]) * adam_chunk(EIGHT) + (threadIdx.x >> 6) * 256;
  if (b >= T.n) return;
  if (T.n - b < 256) {
    adamw_tail<EIGHT>(T, h, b, lane);
    return;
  }
  // one straight body for each combination of types (the same for the whole block)
#define MOE_ADAM_CASE(P32, MASTER)                                              \
  switch (T.flags & (kAdamG32 | kAdam8bit)) {                                   \
    case 0: adamw_run<P32, MASTER, false, false>(T, h, b, lane); break;         \
    case kAdamG32: adamw_run<P32, MASTER, true, false>(T, h, b, lane); break;   \
    case kAdam8bit: adamw_run<P32, MASTER, false, EIGHT>(T, h, b, lane); break; \
    default: adamw_run<P32, MASTER, true, EIGHT>(T, h, b, lane);                \
  }
  if (T.flags & kAdamP32) { MOE_ADAM_CASE(true, false) }
  else if (T.master) { MOE_ADAM_CASE(false, true) }
  else { MOE_ADAM_CASE(false, false) }
#undef MOE_ADAM_CASE
}

namespace {

// Sum of g^2 of one chunk, in 64 bits (no square of an fp32 value overflows or vanishes there).
// Each thread has U loads of 16 bytes in flight; the values behind the last of them go one by one.
// Bound by HBM: 604M bf16 values in 176 us, 6.9 TB/s (4 or 16 loads: 179, 185), and 4 us for the final sum;
// 300M fp32 values in 182 us.
template <bool G32>
__device__ __forceinline__ double square_sum(const void* g, int64_t a, int64_t z) {
  constexpr int V = G32 ? 4 : 8, U = 8;
  double s = 0.0;
  int64_t i = a + threadIdx.x * V;
  const auto add = [&](const u32x4_nt& q) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (G32) {
        const double x = (double)__uint_as_float(q[j]);
        s += x * x;
      } else {
        const double x = (double)lo_bf16(q[j]), y = (double)hi_bf16(q[j]);
        s += x * x;
        s += y * y;
      }
    }
  };
  const char* p = (const char*)g;
  constexpr int kSize = G32 ? 4 : 2;
  for (; i + (U - 1) * 256 * V + V <= z; i += U * 256 * V) {
    u32x4_nt q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) q[u] = __builtin_nontemporal_load((const u32x4_nt*)(p + (i + u * 256 * V) * kSize));
#pragma unroll
    for (int u = 0; u < U; ++u) add(q[u]);
  }
  for (; i < z; i += 256 * V) {
    if (i + V <= z) {
      add(*(const u32x4_nt*)(p + i * kSize));
    } else {
      for (int64_t j = i; j < z; ++j) {
        const double x = G32 ? (double)((const float*)g)[j] : (double)bf16_to_f32(((const uint16_t*)g)[j]);
        s += x * x;
      }
    }
  }
  return s;
}

}  // namespace

__global__ __launch_bounds__(256) void grad_norm_kernel(GradBatch batch, int chunk, double* __restrict__ part) {
  __shared__ double sh[4];
  const int which = tensor_of(batch, blockIdx.x);
  const void* g = batch.g[which];
  const int64_t n = batch.n32[which] >> 1, a = (int64_t)(blockIdx.x - batch.first[which]) * chunk;
  const int64_t z = n - a < chunk ? n : a + chunk;
  double s = batch.n32[which] & 1 ? square_sum<true>(g, a, z) : square_sum<false>(g, a, z);
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

namespace {

constexpr int64_t kMaxChunks = (int64_t)1 << 22;  // blocks a launch: a grid's threads fit 32 bits

// Calls fn(batch, chunks, index of the batch's first tensor) for runs of up to Batch::kMost tensors and
// kMaxChunks chunks of `chunk` values.  A tensor that a launch ends in goes on in the next: its first
// chunk then lies before that launch's.
template <class Batch, class F>
hipError_t for_batches(const moe_tensor* t, int64_t n, int64_t chunk, F fn) {
  Batch b;
  b.n = 0;
  int64_t chunks = 0, first = 0;
  const auto flush = [&]() {
    const hipError_t e = chunks > 0 ? fn(b, chunks, first) : hipSuccess;
    b.n = 0;
    chunks = 0;
    return e;
  };
  for (int64_t i = 0; i < n; ++i) {
    const int64_t all = (t[i].n + chunk - 1) / chunk;
    int64_t done = 0;
    do {
      if (b.n == Batch::kMost || chunks == kMaxChunks) {
        const hipError_t e = flush();
        if (e != hipSuccess) return e;
      }
      if (b.n == 0) first = i;
      b.put(t[i]);
      b.first[b.n++] = (int32_t)(chunks - done);
      const int64_t take = all - done < kMaxChunks - chunks ? all - done : kMaxChunks - chunks;
      done += take;
      chunks += take;
    } while (done < all);
  }
  return flush();
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
  const auto run = [&](const auto& b, int64_t chunks, int64_t first) {
    constexpr bool EIGHT = std::decay_t<decltype(b)>::kEight;
    AdamScalars h = hp;
    h.first_tensor = first;
    adamw_kernel<EIGHT><<<(unsigned)chunks, adam_threads(EIGHT), 0, st>>>(b, h);
    return hipGetLastError();
  };
  bool eight = false;
  for (int64_t i = 0; i < n; ++i) eight |= t[i].n > 0 && t[i].state == MOE_STATE_8BIT;
  return eight ? for_batches<AdamBatch<true>>(t, n, adam_chunk(true), run)
               : for_batches<AdamBatch<false>>(t, n, adam_chunk(false), run);
}

size_t grad_norm_ws_bytes(const moe_tensor* t, int64_t n) { return (size_t)norm_chunks(t, n, norm_chunk(t, n)) * 8; }

hipError_t launch_grad_norm(const moe_tensor* t, int64_t n, float max_norm, float* norm, float* scale, double* part,
                            hipStream_t st) {
  const int64_t chunk = norm_chunk(t, n);
  int64_t at = 0;
  const hipError_t e = for_batches<GradBatch>(t, n, chunk, [&](const GradBatch& b, int64_t chunks, int64_t) {
    grad_norm_kernel<<<(unsigned)chunks, 256, 0, st>>>(b, (int)chunk, part + at);
    at += chunks;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  grad_norm_final_kernel<<<1, 1024, 0, st>>>(part, at, max_norm, norm, scale);
  return hipGetLastError();
}

}  // namespace moe
