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

#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// Blocks of four waves, a token each, that walk the tokens behind (a launch holds at most 2^32 threads).
unsigned token_grid(int T) { return (unsigned)(T < (1 << 24) ? (T + 3) / 4 : 1 << 22); }

// A double of another lane by DPP; lanes that get none keep `old`.
template <int kCtrl, int kRowMask>
__device__ __forceinline__ double dpp64(double old, double v) {
  const int hi = __builtin_amdgcn_update_dpp(__double2hiint(old), __double2hiint(v), kCtrl, kRowMask, 0xf, kRowMask == 0xf);
  const int lo = __builtin_amdgcn_update_dpp(__double2loint(old), __double2loint(v), kCtrl, kRowMask, 0xf, kRowMask == 0xf);
  return __hiloint2double(hi, lo);
}
__device__ __forceinline__ double lane_f64(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane), __builtin_amdgcn_readlane(__double2loint(v), lane));
}
__device__ __forceinline__ double wave_max_f64(double v) {
  v = fmax(v, dpp64<0x128, 0xf>(v, v));
  v = fmax(v, dpp64<0x124, 0xf>(v, v));
  v = fmax(v, dpp64<0x122, 0xf>(v, v));
  v = fmax(v, dpp64<0x121, 0xf>(v, v));
  v = fmax(v, dpp64<0x142, 0xa>(v, v));
  v = fmax(v, dpp64<0x143, 0xc>(v, v));
  return lane_f64(v, 63);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
  v += dpp64<0x128, 0xf>(0.0, v);
  v += dpp64<0x124, 0xf>(0.0, v);
  v += dpp64<0x122, 0xf>(0.0, v);
  v += dpp64<0x121, 0xf>(0.0, v);
  v += dpp64<0x142, 0xa>(0.0, v);
  v += dpp64<0x143, 0xc>(0.0, v);
  return lane_f64(v, 63);
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

// One token by a wave, everything in 64 bits; lane l holds the experts l, l + 64, ... and gets slot l.
struct Slot {
  int id;  // -1: none
  float w;
};
template <int EPL>
__device__ __forceinline__ Slot score_choose_token(const ScoreArgs& p, const float* __restrict__ row,
                                                   const float* __restrict__ bias, double* sh) {
  const int lane = threadIdx.x & 63;
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
  if (__ballot(bad)) return Slot{-1, NAN};
  if (p.groups > 1) {
    const int each = p.E / p.groups;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sh[lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    double b1 = -INFINITY, b2 = -INFINITY;
    if (lane < p.groups) {
#pragma unroll 4
      for (int i = 0; i < each; ++i) {
        const double v = sh[lane * each + i];
        b2 = v > b1 ? b1 : v > b2 ? v : b2;
        b1 = v > b1 ? v : b1;
      }
    }
    const double v = p.group_best == 2 && b2 > -INFINITY ? b1 + b2 : b1;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const double o = lane_f64(v, g);
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
    double best = -INFINITY;
    int at = -1;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (c[i] > best) {  // ids rise with i: a tie keeps the lower one
        best = c[i];
        at = lane + 64 * i;
      }
    const double m = wave_max_f64(best);
    int be = 0x7FFFFFFF;  // the lowest id of those that have the maximum
    for (uint64_t won = __ballot(at >= 0 && best == m); won; won &= won - 1)
      be = min(be, __builtin_amdgcn_readlane(at, __builtin_ctzll(won)));
    if (be == 0x7FFFFFFF) break;  // the same in every lane
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (be == lane + 64 * i) c[i] = -INFINITY;
    if (lane == j) mine = be;
  }
  const bool there = mine >= 0;
  const double q = chosen_weight(p, there, there ? (double)row[mine] : 0.0, top, sum);
  return Slot{mine, (float)(q * p.scale)};
}

// Any shape: one wave per token.
template <int EPL>
__global__ __launch_bounds__(256) void score_choose_kernel(const ScoreArgs p, const float* __restrict__ logits,
                                                           const float* __restrict__ bias,
                                                           const uint8_t* __restrict__ mask, int32_t* __restrict__ ids,
                                                           float* __restrict__ w) {
  __shared__ double sh_c[4][EPL * 64];
  const int wv = threadIdx.x >> 6;
  const int lane = threadIdx.x & 63;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wv; t < p.T; t += (int64_t)gridDim.x * 4) {
    Slot s{-1, 0.0f};
    if (!mask || mask[t] != 0) s = score_choose_token<EPL>(p, logits + t * p.E, bias, sh_c[wv]);
    if (lane < p.k) {
      ids[t * p.k + lane] = s.id;
      w[t * p.k + lane] = s.w;
    }
  }
}

// ------------------------------------------------------------------------------ fast choice
// LPT lanes a token (16: four tokens a wave; 64: one), for k <= 16 and a number of groups that divides
// 16.  Each group's experts lie in the EPL registers of LPT / groups neighbouring lanes.  Scores are
// fp32; a value's lowest four bits are replaced by its register's number, so that it names its expert
// within the lane.  A lane keeps its best four in order, and a round of the choice is one maximum over the
// lanes (in the vector ALU) of their first, whose lane then moves up its others; a lane that has given
// four takes the next four out of its registers.  (With the best two, most rounds of a wave had a lane to
// fill up again: 21804x256 in groups 68 us for the whole call.)  A group's value is made of its best two as they
// were, without register numbers.
//
// An order that fp32 does not settle is found, not guessed, wherever two values that decide something differ
// by less than what scores can be off.  The chosen and the first left out (and no other could be among them: one
// more round shows the next value): their values again in 64 bits, one a lane, and their order by counting.
// The last group that stays and the first that does not, a softmax with a bias (whose sum would have to be
// taken again), or a value that is no ordinary number: the whole token in 64 bits, by the wave.
// (Behind the last expert that can be chosen the rounds find empty places, kNone with a register's number.  They decide
// nothing, however many lanes hold the same, and none of them is a candidate: 16384 tokens, eight of 8 experts 18 us.)
// What a score is off, relative to itself, in u = 2^-24: a sigmoid |x| + 5 (the exponential's argument is rounded,
// which counts |x| (1 - s); the exponential 2, the sum 1, the reciprocal 2), a softmax |x - max| + 5 and a sum of up
// to 16 terms a lane; the addition of the bias 1, and the four bits 16 between two values.  As |s| <= |c| + max |bias|,
// two sigmoids are apart above 2^-18 (64 u) of |c| + max |bias| as long as that is above 1e-6 (x > -14:
// 2 (14 + 5 + 1) + 16), two softmaxes above 2^-16 for values above 1e-30 (69 below the largest).  A group's value v has
// two scores without the four bits, |c1| + |c2| <= |v| + 4 max |bias|: apart above 2^-19 (32 u) of |v| + 6 max |bias|
// as long as that is above 1e-3 (of x below -10 there is then no more than u / 500 in it), for a softmax above 2^-15.
// What is smaller goes to 64 bits.
//
// Tokens that are done again wait until the block's others are through: what they need in registers is then no
// longer kept through the choice (16384x128 22 -> 20 us, 21804x256 in groups 57 -> 52; with four waves a block 49,
// and 39 since a tie is its own token's matter).  Kernels of 21804x256 in groups: choice 28 us, scan 5, places 5.
// What bounds the choice are the chains of a wave's two passes: vector ALU a third of the time (2400 instructions a
// wave), memory and LDS waits half.  Asking for the second pass's logits during the first costs registers: 43 us.
//
// A block takes `seg` tokens, keeps their ids, and gives each pair its rank among the block's pairs of the
// same expert (each wave a share of the pairs, in order; lanes with the same expert by one ballot per id bit)
// and each expert its count: the plan's first pass, without reading the ids back.  A batch that is one
// block's writes the whole plan.
constexpr int kChooseWaves = 4;
constexpr int kSegPairs = 2048;   // pairs of a block, at most
constexpr int kSegments = 1024;   // blocks, at most, that the plan is made of
constexpr int kOneBlock = 32;     // tokens that one block does by itself (64x256: 20 us, 17.7 in two blocks)
constexpr float kNone = -3.0e38f; // below every value that counts: those are above -2 kFarBias
constexpr float kEmpty = -1e38f;  // above a place without an expert (kNone with a register's number), below the others
constexpr float kFarBias = 1e30f; // a finite bias from here on: every token in 64 bits
constexpr int kRedo = -2;         // in the place of a token's ids: to be done again

struct SegPlan {
  int seg, S;  // tokens a block; blocks
};
__host__ __device__ inline SegPlan seg_plan(int64_t T, int64_t k) {
  if (T <= kOneBlock) return SegPlan{kOneBlock, 1};
  const int64_t seg = ((T + kSegments - 1) / kSegments + 31) / 32 * 32;
  return SegPlan{(int)seg, (int)((T + seg - 1) / seg)};
}
bool seg_plan_fits(int64_t T, int64_t k) { return T <= (int64_t)kSegments * kSegPairs && seg_plan(T, k).seg * k <= kSegPairs; }

// Inclusive sum over a wave's lanes, in the vector ALU.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 of each row into the next: rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 into rows 2 and 3
  return v;
}

// By the threads of a block, 256 of which have four experts each: first positions of the experts (start, in LDS, which
// may be the counts themselves) from their counts, to offsets and counts too where they are asked for.
__device__ __forceinline__ void expert_starts(int E, const int32_t* cnt, int* start, int32_t* __restrict__ offsets,
                                              int32_t* __restrict__ counts) {
  __shared__ int part[4];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, e0 = threadIdx.x * 4;
  int c[4], sum = 0, x = 0;
  if (wv < 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += c[i] = e0 + i < E ? cnt[e0 + i] : 0;
    x = wave_scan(sum);
    if (lane == 63) part[wv] = x;
  }
  __syncthreads();
  if (wv < 4) {
    int at = x - sum;
    for (int i = 0; i < wv; ++i) at += part[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e0 + i < E) {
        start[e0 + i] = at;
        if (offsets) offsets[e0 + i] = at;
        if (counts) counts[e0 + i] = c[i];
      }
      at += c[i];
    }
    if (offsets && threadIdx.x == 255) offsets[E] = at;
  }
  __syncthreads();
}

template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
  v = row16_max(v);
  if constexpr (LPT == 64) {
    v = fmaxf(v, dpp<0x142, 0xa>(v, v));
    v = fmaxf(v, dpp<0x143, 0xc>(v, v));
    v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
  return LPT == 64 ? wave_sum_dpp(v) : row16_sum(v);
}

// e^(x - m), finite x and m, with the difference's rounding put back: from |x - m| = 64 on that alone is 2^-18.
__device__ __forceinline__ float exp_apart(float x, float m) {
  const float d = x - m, t = d - x, rest = (x - (d - t)) - (m + t), e = expf(d);
  return fmaf(e, rest, e);
}

// Exchange with the lane whose number differs in the bit `of`, or (in a row, once pairs agree) the mirror image.
template <int kOf>
__device__ __forceinline__ float partner(float v) {
  if constexpr (kOf == 1) return dpp<0xB1, 0xf>(v, v);        // quad_perm 1 0 3 2
  else if constexpr (kOf == 2) return dpp<0x4E, 0xf>(v, v);   // quad_perm 2 3 0 1
  else if constexpr (kOf == 4) return dpp<0x141, 0xf>(v, v);  // row_half_mirror
  else if constexpr (kOf == 8) return dpp<0x140, 0xf>(v, v);  // row_mirror
  else return __shfl_xor(v, kOf, 64);
}
template <int kOf>
__device__ __forceinline__ void merge_best(float& a, float& b) {
  const float c = partner<kOf>(a), d = partner<kOf>(b);
  b = fmaxf(fminf(a, c), fmaxf(b, d));
  a = fmaxf(a, c);
}

// Groups of kLg lanes of a row of 16: how many have a larger value, or the same and a lower number.
template <int kLg, int kRot = kLg>
__device__ __forceinline__ void rank_groups(float v, int& rank) {
  if constexpr (kRot < 16) {
    const float o = dpp<0x120 + kRot, 0xf>(v, v);  // the lane kRot below, around the row
    rank += o > v || (o == v && ((int)threadIdx.x & 15) >= kRot);
    rank_groups<kLg, kRot + kLg>(v, rank);
  }
}

// Places of 16 lanes' values in descending order; equal ones by id.  near: another value within 2^-40, but not equal.
template <int kRot>
__device__ __forceinline__ void rank_candidates(double v, int id, int& rank, bool& near) {
  if constexpr (kRot < 16) {
    auto turn = [](int w) __attribute__((always_inline)) {
      return __builtin_amdgcn_update_dpp(w, w, 0x120 + kRot, 0xf, 0xf, true);
    };
    const double o = __hiloint2double(turn(__double2hiint(v)), turn(__double2loint(v)));
    const int oid = turn(id);
    rank += o > v || (o == v && oid < id);
    near |= o != v && fabs(o - v) < 0x1p-40;
    rank_candidates<kRot + 1>(v, id, rank, near);
  }
}

template <int LPT, int EPL, int EPL64, bool SIG>
__global__ __launch_bounds__(64 * kChooseWaves, LPT == 16 ? 3 : 2) void score_choose_fast_kernel(
    const ScoreArgs p, const float* __restrict__ logits, const float* __restrict__ bias, const uint8_t* __restrict__ mask,
    int32_t* __restrict__ ids, float* __restrict__ w, int seg, int32_t* __restrict__ segcnt, uint16_t* __restrict__ ranks,
    int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ perm, int32_t* __restrict__ inv_perm) {
  constexpr int NW = kChooseWaves, NT = 64 * NW, TPW = 64 / LPT;  // waves, threads, tokens a wave and pass
  __shared__ double sh_c[NW][EPL64 * 64];
  __shared__ int sh_ids[kSegPairs], sh_cand[NW][TPW][16];
  extern __shared__ int sh_run[];  // [NW][E], where the plan is made here
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, sub = lane / LPT, l = lane % LPT;
  const int lg = LPT / p.groups, each = p.E / p.groups, grp = l / lg;
  const int epl = (each + lg - 1) / lg, first = (l % lg) * epl, n = max(min(each - first, epl), 0), base = grp * each + first;
  const bool vec = p.E % 4 == 0 && each % 4 == 0 && epl % 4 == 0;
  const int64_t t0 = (int64_t)blockIdx.x * seg;
  const int ntok = (int)min((int64_t)seg, p.T - t0);

  // the biases; a register without an expert reads its neighbour's and is barred as by a bias of -inf
  float b[EPL], bm = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) b[i] = bias ? bias[min(base + i, p.E - 1)] : 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (fabsf(b[i]) < INFINITY) bm = fmaxf(bm, fabsf(b[i]));
    if (b[i] == -INFINITY || i >= n) b[i] = kNone;
  }
  bm = lanes_max<LPT>(bm);
  const bool far = bm >= kFarBias;

  for (int r0 = wv * TPW; r0 < ntok; r0 += NW * TPW) {
    const int local = r0 + sub;
    const int64_t t = t0 + min(local, ntok - 1);
    const bool active = local < ntok && (!mask || mask[t] != 0);
    const float* row = logits + t * p.E;
    float x[EPL], c[EPL];
    if (vec) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4) {
        const float4 v = *(const float4*)(row + min(base + i, p.E - 4));
        x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) x[i] = row[min(base + i, p.E - 1)];
    }
    float top = 0.0f, sum = 1.0f, inv = 1.0f;
    if constexpr (!SIG) {
      top = x[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) top = fmaxf(top, x[i]);  // (a neighbour's logit counts once more: no matter)
      top = lanes_max<LPT>(top);
      if (top == -INFINITY) top = 0.0f;
      sum = 0.0f;
      int here = n;
      asm volatile("" : "+v"(here));  // compared where it is needed: 16 masks would fill the scalar registers
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        c[i] = __expf(x[i] - top);
        if (i < here) sum += c[i];
      }
      sum = lanes_sum<LPT>(sum);
      inv = 1.0f / sum;
    }
    float nought = 0.0f;  // NaN once a value is no ordinary number
    float b1 = kNone, b2 = kNone, b3 = kNone, b4 = kNone, g1 = kNone, g2 = kNone;
    auto insert = [&](float v) __attribute__((always_inline)) {
      b4 = __builtin_amdgcn_fmed3f(b3, b4, v);
      b3 = __builtin_amdgcn_fmed3f(b2, b3, v);
      b2 = __builtin_amdgcn_fmed3f(b1, b2, v);
      b1 = fmaxf(b1, v);
    };
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float v = (SIG ? __builtin_amdgcn_rcpf(1.0f + __expf(-x[i])) : c[i] * inv) + b[i];
      const bool barred = x[i] == -INFINITY;
      nought = fmaf(barred ? b[i] : v, 0.0f, nought);
      const float u = barred ? kNone : v;
      g2 = __builtin_amdgcn_fmed3f(g1, g2, u);
      g1 = fmaxf(g1, u);
      c[i] = __uint_as_float((__float_as_uint(u) & ~15u) | (15 - i));
      insert(c[i]);
    }
    bool odd = far || !(nought == 0.0f);  // something for the 64-bit path
    constexpr float kOff = SIG ? 0x1p-18f : 0x1p-16f, kGroupOff = SIG ? 0x1p-19f : 0x1p-15f;
    bool dropped = false;
    if (p.groups > 1) {
      if (lg >= 2) merge_best<1>(g1, g2);
      if (lg >= 4) merge_best<2>(g1, g2);
      if (lg >= 8) merge_best<4>(g1, g2);
      if (LPT == 64 && lg >= 16) merge_best<8>(g1, g2);
      if (LPT == 64 && lg >= 32) merge_best<16>(g1, g2);
      const bool alive = g1 > kEmpty;
      const float v = p.group_best == 2 && g2 > kEmpty ? g1 + g2 : g1;
      int rank = 0;
      if constexpr (LPT == 16) {
        if (lg == 1) rank_groups<1>(v, rank);
        else if (lg == 2) rank_groups<2>(v, rank);
        else if (lg == 4) rank_groups<4>(v, rank);
        else rank_groups<8>(v, rank);
      } else {
        for (int g = 0; g < p.groups; ++g) {
          const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), g * lg));
          rank += o > v || (o == v && g < grp);
        }
      }
      dropped = !alive || rank >= p.group_topk;
      const float least = -lanes_max<LPT>(dropped ? kNone : -v), next = lanes_max<LPT>(dropped && alive ? v : kNone);
      const float near = fabsf(next) + 6 * bm;
      odd |= next > kEmpty && !(least - next > kGroupOff * near && (!SIG || near > 1e-3f));
      if (dropped) b1 = b2 = b3 = b4 = kNone;
    }
    if (!active) b1 = kNone - 1e35f * l;  // one winner in every round, which takes nothing
    const int keep = min(p.k + 1, 16);    // candidates: one more than are chosen, where the lanes hold it
    int* cand = sh_cand[wv][sub];
    float mine_v = 0.0f, last = 0.0f;     // lane j: the value of round j; the last round's
    int given = 0;
    bool several = false;                 // winners in a round
    for (int j = 0; j <= keep; ++j) {
      const float m = lanes_max<LPT>(b1);
      const bool win = b1 == m;
      const uint64_t won = __ballot(win);
      if (__popcll(won) != TPW) several |= m > kEmpty && (LPT == 64 || __popcll(won >> (16 * sub) & 0xFFFF) != 1);
      last = m;
      if (j == keep) break;
      if (l == j) mine_v = m;
      if (win && active) {
        cand[j] = base + 15 - (int)(__float_as_uint(m) & 15u);
        b1 = b2;
        b2 = b3;
        b3 = b4;
        b4 = kNone;
        ++given;
      }
      if constexpr (EPL > 4) {
        if (__ballot(given == 4)) {
          const float a1 = b1, a2 = b2, a3 = b3, a4 = b4;
          b1 = b2 = b3 = b4 = kNone;
#pragma unroll
          for (int i = 0; i < EPL; ++i) insert(c[i] < m && !dropped ? c[i] : kNone);
          if (given == 4) {
            given = 0;
          } else {
            b1 = a1, b2 = a2, b3 = a3, b4 = a4;
          }
        }
      }
    }
    // what follows each candidate (the last: the value of the round behind it), and whether it is apart from it
    float after = __uint_as_float(
        __builtin_amdgcn_update_dpp(__float_as_uint(last), __float_as_uint(mine_v), 0x101, 0xf, 0xf, false));
    if (l == keep - 1) after = last;
    auto apart = [&](float hi, float lo) __attribute__((always_inline)) { return hi - lo > kOff * (fabsf(lo) + bm); };
    const bool unsure = active && l < p.k && !apart(mine_v, after);
    odd |= several || (active && l < p.k && !(fabsf(mine_v) + (SIG ? bm : 0.0f) > (SIG ? 1e-6f : 1e-30f) && mine_v > kEmpty));
    if (!SIG && bias) odd |= unsure;
    odd |= active && l == p.k - 1 && !apart(mine_v, last);
    // the lanes' candidates (an id past the experts: none was left, and the token is done again below)
    int mine = active && l < keep ? min(cand[l], p.E - 1) : 0;
    if ((SIG || !bias) && __ballot(unsure)) {
      // (a round in which nothing was left has no candidate, whatever its winner was)
      const bool real = active && l < keep && mine_v > kEmpty;
      double v = -INFINITY;
      if (real) {
        const double x1 = row[mine];
        v = SIG ? sigmoid_scaled(x1, 0.0) + (bias ? (double)bias[mine] : 0.0) : x1;
      }
      int rank = 0;
      bool near = false;
      rank_candidates<1>(v, mine, rank, near);
      if constexpr (!SIG) odd |= near && real;  // logits whose scores may be equal in 64 bits
      if (real) cand[rank] = mine;
      if (real) mine = min(cand[l], p.E - 1);
    }
    // slot l of the lanes' token, and its weight
    const bool slot = l < p.k && local < ntok;
    int id = -1;
    float q = 0.0f;
    if (slot && active) id = mine;
    const float x1 = id >= 0 ? row[id] : 0.0f;
    float z;
    if constexpr (SIG) {
      const float m = p.renorm ? lanes_max<LPT>(id >= 0 ? fminf(x1, 0.0f) : -INFINITY) : 0.0f;
      z = id >= 0 ? exp_apart(fminf(x1, 0.0f), m) / (1.0f + expf(-fabsf(x1))) : 0.0f;
      if (p.renorm) z /= lanes_sum<LPT>(z);
    } else {
      const float m = p.renorm ? lanes_max<LPT>(id >= 0 ? x1 : -INFINITY) : top;
      z = id >= 0 ? exp_apart(x1, m) : 0.0f;
      z /= p.renorm ? lanes_sum<LPT>(z) : sum;
    }
    q = active ? z * p.scale : 0.0f;
    // (a token that is done again gets its ids below)
    const uint64_t again = __ballot(odd && active);
    const bool redo = LPT == 64 ? again != 0 : (again >> (16 * sub) & 0xFFFF) != 0;
    if (slot) {
      if (!redo) {
        ids[t * p.k + l] = id;
        w[t * p.k + l] = q;
      }
      sh_ids[local * p.k + l] = redo ? kRedo : id;
    }
  }
  __builtin_amdgcn_wave_barrier();
  // The tokens that are done again: after the others, so that what these need in registers is not kept meanwhile.
  for (int r0 = wv * TPW; r0 < ntok; r0 += NW * TPW) {
    uint64_t again = __ballot(l == 0 && r0 + sub < ntok && sh_ids[min(r0 + sub, ntok - 1) * p.k] == kRedo);
    while (again) {
      const int local = r0 + __builtin_ctzll(again) / LPT;
      again &= again - 1;
      const int64_t t = t0 + local;
      const Slot s = score_choose_token<EPL64>(p, logits + t * p.E, bias, sh_c[wv]);
      if (lane < p.k) {
        ids[t * p.k + lane] = s.id;
        w[t * p.k + lane] = s.w;
        sh_ids[local * p.k + lane] = s.id;
      }
    }
  }
  if (!segcnt && !perm) return;  // the plan is made elsewhere

  // ------------------------------------------------------------------ ranks and counts
  constexpr int STEPS = kSegPairs / NT;
  const int pairs = ntok * p.k, share = ((pairs + NW - 1) / NW + 63) / 64 * 64;
  const int lo = min(wv * share, pairs), hi = min(lo + share, pairs);
  int* run = sh_run + wv * p.E;
  for (int e = lane; e < p.E; e += 64) run[e] = 0;
  __syncthreads();
  int bits = 1;
  while ((1 << bits) < p.E) ++bits;
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  int of[STEPS], rank[STEPS];  // the lane's pairs: expert, rank in the wave's share
#pragma unroll
  for (int u = 0; u < STEPS; ++u) {
    of[u] = -1;
    rank[u] = 0;
    if (lo + 64 * u >= hi) continue;
    const int i = lo + 64 * u + lane, e = i < hi ? sh_ids[i] : -1;
    uint64_t same = __ballot(e >= 0);
    for (int x = 0; x < bits; ++x) {
      const uint64_t set = __ballot((e >> x) & 1);
      same &= (e >> x) & 1 ? set : ~set;
    }
    if (e >= 0) rank[u] = run[e] + __popcll(same & below);
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && (same & below) == 0) run[e] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
    of[u] = e;
  }
  __syncthreads();
  int* start = (int*)sh_c;  // first positions of the experts, where the block is the whole batch
  for (int e = threadIdx.x; e < p.E; e += NT) {
    int at = 0;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      const int c = sh_run[v * p.E + e];
      sh_run[v * p.E + e] = at;
      at += c;
    }
    if (perm) start[e] = at;  // the total, turned into first positions below
    else segcnt[(int64_t)blockIdx.x * p.E + e] = at;
  }
  __syncthreads();
  if (perm) expert_starts(p.E, start, start, offsets, counts);
#pragma unroll
  for (int u = 0; u < STEPS; ++u) {
    const int i = lo + 64 * u + lane;
    if (i >= hi) break;
    const int at = of[u] >= 0 ? run[of[u]] + rank[u] : 0;
    if (!perm) {
      ranks[t0 * p.k + i] = (uint16_t)at;
    } else if (of[u] >= 0) {
      perm[start[of[u]] + at] = i;
      inv_perm[i] = start[of[u]] + at;
    } else {
      inv_perm[i] = -1;
    }
  }
}

// Each expert's counts over the blocks: exclusive sums in their place, the total in counts.  16 experts a
// block (64 bytes of a row); 64 groups of neighbouring rows.
__global__ __launch_bounds__(1024) void score_scan_kernel(int32_t* __restrict__ segcnt, int E, int S,
                                                          int32_t* __restrict__ counts) {
  __shared__ int part[64][16];
  const int l = threadIdx.x & 15, grp = threadIdx.x >> 4, e = blockIdx.x * 16 + l;
  constexpr int ROWS = kSegments / 64;
  const int per = (S + 63) / 64, lo = grp * per;
  int v[ROWS], sum = 0;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    v[i] = i < per && lo + i < S && e < E ? segcnt[(int64_t)(lo + i) * E + e] : 0;
    sum += v[i];
  }
  part[grp][l] = sum;
  __syncthreads();
  if (threadIdx.x < 256) {  // the groups' sums, in place: 16 threads an expert, four groups each
    const int x = threadIdx.x & 15, q = threadIdx.x >> 4;
    int s4[4], t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s4[i] = t;
      t += part[4 * x + i][q];
    }
    int y = t;
    y += __builtin_amdgcn_update_dpp(0, y, 0x111, 0xf, 0xf, true);
    y += __builtin_amdgcn_update_dpp(0, y, 0x112, 0xf, 0xf, true);
    y += __builtin_amdgcn_update_dpp(0, y, 0x114, 0xf, 0xf, true);
    y += __builtin_amdgcn_update_dpp(0, y, 0x118, 0xf, 0xf, true);
#pragma unroll
    for (int i = 0; i < 4; ++i) part[4 * x + i][q] = y - t + s4[i];
    if (x == 15 && blockIdx.x * 16 + q < E) counts[blockIdx.x * 16 + q] = y;
  }
  __syncthreads();
  if (e >= E) return;
  int at = part[grp][l];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    if (i < per && lo + i < S) {
      segcnt[(int64_t)(lo + i) * E + e] = at;
      at += v[i];
    }
}

// Positions of the pairs: the expert's first, its pairs in the blocks before, the rank in the block.
__global__ __launch_bounds__(256) void score_place_kernel(const int32_t* __restrict__ ids, int64_t pairs, int E, int seg_pairs,
                                                          const int32_t* __restrict__ segbase,
                                                          const uint16_t* __restrict__ ranks,
                                                          const int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                          int32_t* __restrict__ perm, int32_t* __restrict__ inv_perm) {
  __shared__ int start[1024];
  constexpr int PER = 2;
  int e[PER], at[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t q = (int64_t)blockIdx.x * (256 * PER) + 256 * i + threadIdx.x;
    e[i] = q < pairs ? ids[q] : -1;
    at[i] = q < pairs ? ranks[q] : 0;
    if (e[i] >= 0) at[i] += segbase[q / seg_pairs * E + e[i]];
  }
  expert_starts(E, counts, start, blockIdx.x == 0 ? offsets : nullptr, nullptr);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t q = (int64_t)blockIdx.x * (256 * PER) + 256 * i + threadIdx.x;
    if (q >= pairs) return;
    const int pos = e[i] >= 0 ? start[e[i]] + at[i] : -1;
    if (pos >= 0) perm[pos] = (int32_t)q;
    inv_perm[q] = pos;
  }
}

namespace {

// The plan's tables: counts of the segments, ranks of the pairs.
size_t seg_ws_bytes(int64_t T, int64_t E, int64_t k) {
  const SegPlan sp = seg_plan(T, k);
  return sp.S == 1 ? 0 : (size_t)sp.S * E * sizeof(int32_t) + (size_t)T * k * sizeof(uint16_t);
}

// Registers a lane needs for its experts, at 16 and at 64 lanes a token
int lane_share(const ScoreArgs& p, int lpt) {
  const int lg = lpt / p.groups, each = p.E / p.groups;
  return (each + lg - 1) / lg;
}

bool is_fast(const ScoreArgs& p) { return p.k <= 16 && 16 % p.groups == 0 && lane_share(p, 64) <= 16; }

struct RouteOut {
  int32_t* ids;
  float* w;
  int32_t *counts, *offsets, *perm, *inv_perm;
};

template <int LPT, int EPL, int EPL64>
void launch_fast(const ScoreArgs& p, const float* logits, const float* bias, const uint8_t* mask, const RouteOut& o,
                 const SegPlan& sp, int32_t* segcnt, uint16_t* ranks, hipStream_t st) {
  const size_t lds = kChooseWaves * (size_t)p.E * sizeof(int);
  const unsigned block = 64 * kChooseWaves;
  int32_t* perm = sp.S == 1 && o.perm ? o.perm : nullptr;
  const unsigned grid = (unsigned)sp.S;
  if (p.sigmoid)
    score_choose_fast_kernel<LPT, EPL, EPL64, true><<<grid, block, lds, st>>>(p, logits, bias, mask, o.ids, o.w, sp.seg, segcnt,
                                                                           ranks, o.counts, o.offsets, perm, o.inv_perm);
  else
    score_choose_fast_kernel<LPT, EPL, EPL64, false><<<grid, block, lds, st>>>(p, logits, bias, mask, o.ids, o.w, sp.seg, segcnt,
                                                                            ranks, o.counts, o.offsets, perm, o.inv_perm);
}

}  // namespace

size_t score_ws_bytes(int64_t T, int64_t E, int64_t k) {
  const size_t a = plan_ws_bytes(T * k, E), b = seg_plan_fits(T, k) ? seg_ws_bytes(T, E, k) : 0;
  return a > b ? a : b;
}

hipError_t launch_score_route(const ScoreArgs& p, const float* logits, const float* bias, const uint8_t* mask,
                              int32_t* ids, float* w, int32_t* counts, int32_t* offsets, int32_t* perm,
                              int32_t* inv_perm, void* ws, hipStream_t st) {
  const int64_t pairs = (int64_t)p.T * p.k;
  if (p.T > 0 && is_fast(p)) {
    const bool here = seg_plan_fits(p.T, p.k);
    SegPlan sp = seg_plan(p.T, p.k);
    if (!here) sp = SegPlan{kSegPairs / p.k, (int)(((int64_t)p.T + kSegPairs / p.k - 1) / (kSegPairs / p.k))};
    int32_t* segcnt = here && sp.S > 1 ? (int32_t*)ws : nullptr;
    uint16_t* ranks = (uint16_t*)(segcnt ? segcnt + (size_t)sp.S * p.E : nullptr);
    const RouteOut o{ids, w, counts, offsets, here ? perm : nullptr, inv_perm};
    const int n16 = lane_share(p, 16);
    // a wave for each token: all its lanes for one (1x256 7.1 us instead of 7.9, in groups 7.8 instead of 8.5; no
    // gain where 16 lanes have eight experts each: 2x128 7.3 and 7.2)
    if (p.T <= kChooseWaves && n16 > 8 && lane_share(p, 64) <= 4)
      launch_fast<64, 4, 4>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    else if (n16 <= 4) launch_fast<16, 4, 1>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    else if (n16 <= 8) launch_fast<16, 8, 2>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    else if (n16 <= 16) launch_fast<16, 16, 4>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    else if (lane_share(p, 64) <= 8) launch_fast<64, 8, 8>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    else launch_fast<64, 16, 16>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    if (segcnt) {
      score_scan_kernel<<<(p.E + 15) / 16, 1024, 0, st>>>(segcnt, p.E, sp.S, counts);
      score_place_kernel<<<(unsigned)((pairs + 511) / 512), 256, 0, st>>>(ids, pairs, p.E, sp.seg * p.k, segcnt, ranks,
                                                                            counts, offsets, perm, inv_perm);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || here) return e;
  } else if (p.T > 0) {
    const dim3 grid(token_grid(p.T)), block(256);
    if (p.E <= 64) score_choose_kernel<1><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    else if (p.E <= 128) score_choose_kernel<2><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    else if (p.E <= 256) score_choose_kernel<4><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    else if (p.E <= 512) score_choose_kernel<8><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    else score_choose_kernel<16><<<grid, block, 0, st>>>(p, logits, bias, mask, ids, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_plan(ids, pairs, p.E, counts, offsets, perm, inv_perm, ws, st);
}

// -------------------------------------------------------------------------------- backward
// One wave per token; lane j < k holds slot j, and the lanes then write the row.
//
// A softmax that is not renormalised subtracts: d_e = s_e (G_e - sum_i g_i s_i) with G_e the g of e's slots.  Of a confident
// token s_e is near 1 and the difference what the other experts leave, so it is taken in 64 bits, of scores whose sum
// is 64-bit too and whose chosen terms are 64-bit exponentials.  The others' are fp32 ones, |x - max| + 2 units of
// 2^-24 each, and that is the difference's relative error (with fp32 sums it was 2^-7 where the others have 2e-5).
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
    bool first = there;  // the lowest of the slots with this id: its term of the sum in 64 bits
    for (int j = 0; j < p.k; ++j) first = first && (__builtin_amdgcn_readlane(id, j) != id || j >= lane);
    float xmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      x[i] = e < p.E ? row[e] : -INFINITY;
      xmax = fmaxf(xmax, x[i]);
    }
    top = wave_max_f64(xmax);
    double part = first ? exp(l - top) - (double)expf((float)l - (float)top) : 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) part += x[i] = expf(x[i] - (float)top);
    sum = wave_sum_f64(part);
  }
  const double q = chosen_weight(p, there, l, top, sum);
  const double dot = p.renorm || dense ? wave_sum_f64(g * q) : 0.0;
  // what slot j adds at its expert, and there the sum over the slots with this id
  const float v = there && !dense ? (float)(p.sigmoid ? (g - dot) * q * sigmoid_scaled(-l, 0.0) : (g - dot) * q) : 0.0f;
  float all = 0.0f;
  double all_g = 0.0;
  for (int j = 0; j < p.k; ++j) {
    const bool same = __builtin_amdgcn_readlane(id, j) == id;
    const float u = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), j));
    const double u_g = lane_f64(g, j);
    if (same) all += u, all_g += u_g;
  }
  if (dense) all = (float)((all_g - dot) * q);
  const float off = dense ? (float)(dot / sum) : 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) out[i] = dense ? -off * x[i] : 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float u = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(all), j));
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e == lane + 64 * i) out[i] = u;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e < p.E) d[e] = out[i];
  }
}

template <int EPL>
__global__ __launch_bounds__(256) void score_backward_kernel(const ScoreArgs p, const float* __restrict__ logits,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ d_w, float* __restrict__ d) {
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < p.T; t += (int64_t)gridDim.x * 4)
    score_backward_token<EPL>(p, logits + t * p.E, ids + t * p.k, d_w + t * p.k, d + t * p.E);
}

// For k <= 16: four tokens a wave, a row of 16 lanes each, lane j with slot j.  The chosen experts' values are made in
// 64 bits as above, once for four tokens; the wave's four rows of the gradient, which lie behind one another, are laid out in
// LDS and written in one piece, 16 bytes a lane, whatever E is.  A softmax that is not renormalised goes through
// LDS too: its rows' exponentials lie where the gradient comes to lie.  An id that occurs twice in a token gets
// the sum in slot order, the same in each of its lanes.  21804x256, sigmoid: 8.5 us where the bytes take 4.8 (one token a
// wave, written 4 bytes a lane: 18); what is left is two dependent loads (ids, then logits) before the first store.
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ double row16_max_f64(double v) {
  v = fmax(v, dpp64<0x128, 0xf>(v, v));
  v = fmax(v, dpp64<0x124, 0xf>(v, v));
  v = fmax(v, dpp64<0x122, 0xf>(v, v));
  return fmax(v, dpp64<0x121, 0xf>(v, v));
}
__device__ __forceinline__ double row16_sum_f64(double v) {
  v += dpp64<0x128, 0xf>(0.0, v);
  v += dpp64<0x124, 0xf>(0.0, v);
  v += dpp64<0x122, 0xf>(0.0, v);
  return v + dpp64<0x121, 0xf>(0.0, v);
}

template <bool SIG, bool DENSE>
__global__ __launch_bounds__(256) void score_backward_rows_kernel(const ScoreArgs p, const float* __restrict__ logits,
                                                                  const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ d_w, float* __restrict__ d) {
  extern __shared__ __attribute__((aligned(16))) float sh_rows[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, sub = lane >> 4, l = lane & 15;
  float* rows = sh_rows + (int64_t)wv * 4 * p.E;
  float* mine = rows + sub * p.E;
  const int64_t waves = blockDim.x / 64;
  for (int64_t t0 = (blockIdx.x * waves + wv) * 4; t0 < p.T; t0 += gridDim.x * waves * 4) {
    const int ntok = (int)min((int64_t)4, p.T - t0), words = ntok * p.E;
    const int64_t t = t0 + min(sub, ntok - 1);
    const float* row = logits + t * p.E;
    const int id = l < p.k ? ids[t * p.k + l] : -1;
    const bool there = id >= 0 && id < p.E;
    const double g = there ? (double)d_w[t * p.k + l] * p.scale : 0.0;
    const double x = there ? (double)row[id] : 0.0;
    double m = 0.0, sum = DENSE ? 0.0 : 1.0;
    if constexpr (DENSE) {
      float xmax = -INFINITY;
      for (int i = 4 * lane; i < words; i += 256) {
        if (i + 4 <= words) {
          *(f32x4*)(rows + i) = *(const f32x4_u*)(logits + t0 * p.E + i);
        } else {
          for (int e = i; e < words; ++e) rows[e] = logits[t0 * p.E + e];
        }
      }
      __builtin_amdgcn_wave_barrier();
      if (sub < ntok) {
#pragma unroll 4
        for (int e = l; e < p.E; e += 16) xmax = fmaxf(xmax, mine[e]);
      }
      xmax = row16_max(xmax);
      m = xmax;
      if (sub < ntok) {
#pragma unroll 4
        for (int e = l; e < p.E; e += 16) sum += mine[e] = expf(mine[e] - xmax);
      }
    } else {
      for (int i = 4 * lane; i < 4 * p.E; i += 256) *(f32x4*)(rows + i) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (p.renorm) m = row16_max_f64(there ? (SIG ? fmin(x, 0.0) : x) : -INFINITY);
    }
    __builtin_amdgcn_wave_barrier();
    double q = there ? (SIG ? sigmoid_scaled(x, m) : exp(x - m)) : 0.0;
    if constexpr (DENSE) {
      bool first = there;  // the lowest of the slots with this id: its term of the sum in 64 bits
      for (int j = 0; j < p.k; ++j) first = first && (__shfl(id, j, 16) != id || j >= l);
      if (first) sum += q - (double)mine[id];
      sum = row16_sum_f64(sum);
    }
    if (p.renorm) sum = row16_sum_f64(q);
    q = there ? q / sum : 0.0;
    const double dot = p.renorm || DENSE ? row16_sum_f64(g * q) : 0.0;
    typedef typename std::conditional<DENSE, double, float>::type part_t;
    part_t v = 0, total = 0;  // the slot's part of the gradient (DENSE: g); over the slots with this id
    if (DENSE) v = g;
    else if (there) v = (part_t)(SIG ? (g - dot) * q * sigmoid_scaled(-x, 0.0) : (g - dot) * q);
    for (int j = 0; j < p.k; ++j) {
      const part_t o = __shfl(v, j, 16);
      if (__shfl(id, j, 16) == id) total += o;
    }
    float all = (float)total;
    if constexpr (DENSE) {
      const float off = (float)(dot / sum);
      const bool any = (__ballot(there) >> (16 * sub) & 0xFFFF) != 0;
      all = (float)((total - dot) * q);
      __builtin_amdgcn_wave_barrier();
      if (sub < ntok) {
#pragma unroll 4
        for (int e = l; e < p.E; e += 16) mine[e] = any ? -off * mine[e] : 0.0f;
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (there && sub < ntok) mine[id] = all;
    __builtin_amdgcn_wave_barrier();
    float* out = d + t0 * p.E;
    for (int i = 4 * lane; i < words; i += 256) {
      if (i + 4 <= words) {
        *(f32x4_u*)(out + i) = *(const f32x4*)(rows + i);
      } else {
        for (int e = i; e < words; ++e) out[e] = rows[e];
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

hipError_t launch_score_backward(const ScoreArgs& p, const float* logits, const int32_t* ids, const float* d_w,
                                 float* d_logits, hipStream_t st) {
  if (p.k <= 16) {
    const int waves = p.T <= 4096 ? 1 : 4;  // few tokens: a wave a block, on as many compute units
    const dim3 grid((token_grid(p.T) + waves - 1) / waves), block(64 * waves);
    const size_t lds = waves * 4 * (size_t)p.E * sizeof(float);
    if (p.sigmoid) score_backward_rows_kernel<true, false><<<grid, block, lds, st>>>(p, logits, ids, d_w, d_logits);
    else if (p.renorm) score_backward_rows_kernel<false, false><<<grid, block, lds, st>>>(p, logits, ids, d_w, d_logits);
    else score_backward_rows_kernel<false, true><<<grid, block, lds, st>>>(p, logits, ids, d_w, d_logits);
    return hipGetLastError();
  }
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
