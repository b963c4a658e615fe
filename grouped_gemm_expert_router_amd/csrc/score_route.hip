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
// fp32; a score's lowest four bits are replaced by its register's number, so that a value names its
// expert within the lane, and a round of the choice is one maximum over the lanes (in the vector ALU) of
// each lane's best, the winner moving up its second best.  The lanes' best two are what a group's value
// is made of as well.
//
// An order that fp32 does not settle is found, not guessed: wherever two values that decide something
// (neighbours in the order up to the first that is left out, the last group that stays and the first that
// does not) differ by less than what scores can be off, or where a value is not an ordinary number, the token
// is done again in 64 bits by the whole wave.  What a score is off, relative to |c| + max |bias|: sigmoid
// 4 2^-24 (an exponential with its argument's rounding, a sum, a reciprocal: |x| s (1 - s) < 1/4), softmax 2^-18
// (logits up to 60 below the largest), and 2^-20 for the four bits; twice that for two values: below 2^-18
// and 2^-16.  About one token in a hundred (256 experts) is done again.
//
// A block takes `seg` tokens, keeps their ids, and gives each pair its rank among the block's pairs of the
// same expert (each wave a quarter of the pairs, in order; lanes with the same expert by one ballot per id
// bit) and each expert its count: the plan's first pass, without reading the ids back.  A batch that is one
// block's writes the whole plan.
constexpr int kSegPairs = 2048;   // pairs of a block, at most
constexpr int kSegments = 512;    // blocks, at most, that the plan is made of
constexpr int kOneBlock = 64;     // tokens that one block does by itself
constexpr float kNone = -3.0e38f; // below every value that counts

struct SegPlan {
  int seg, S;  // tokens a block; blocks
};
__host__ __device__ inline SegPlan seg_plan(int64_t T, int64_t k) {
  if (T <= kOneBlock) return SegPlan{kOneBlock, 1};
  const int64_t seg = ((T + kSegments - 1) / kSegments + 15) / 16 * 16;
  return SegPlan{(int)seg, (int)((T + seg - 1) / seg)};
}
bool seg_plan_fits(int64_t T, int64_t k) { return T <= (int64_t)kSegments * kSegPairs && seg_plan(T, k).seg * k <= kSegPairs; }

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

template <int kRot>
__device__ __forceinline__ void rank_by_rotation(float v, int grp, int lg, int& rank) {
  if constexpr (kRot < 16) {
    const float o = dpp<0x120 + kRot, 0xf>(v, v);  // the lane kRot below, around the row
    const int og = (((int)threadIdx.x - kRot) & 15) / lg;
    rank += o > v || (o == v && og < grp);
    rank_by_rotation<kRot + 1>(v, grp, lg, rank);
  }
}

template <int LPT, int EPL, int EPL64, bool SIG>
__global__ __launch_bounds__(256) void score_choose_fast_kernel(const ScoreArgs p, const float* __restrict__ logits,
                                                                const float* __restrict__ bias,
                                                                const uint8_t* __restrict__ mask,
                                                                int32_t* __restrict__ ids, float* __restrict__ w, int seg,
                                                                int32_t* __restrict__ segcnt, uint16_t* __restrict__ ranks,
                                                                int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ perm, int32_t* __restrict__ inv_perm) {
  constexpr int TPW = 64 / LPT;  // tokens a wave and pass
  __shared__ double sh_c[4][EPL64 * 64];
  __shared__ int sh_ids[kSegPairs];
  extern __shared__ int sh_cnt[];  // [4][E], where the plan is made here
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, sub = lane / LPT, l = lane % LPT;
  const int lg = LPT / p.groups, each = p.E / p.groups, grp = l / lg;
  const int epl = (each + lg - 1) / lg, first = (l % lg) * epl, n = max(min(each - first, epl), 0), base = grp * each + first;
  const bool vec = p.E % 4 == 0 && each % 4 == 0 && epl % 4 == 0;
  const int64_t t0 = (int64_t)blockIdx.x * seg;
  const int ntok = (int)min((int64_t)seg, p.T - t0);

  float b[EPL], bm = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    b[i] = i < n ? (bias ? bias[base + i] : 0.0f) : -INFINITY;
    if (fabsf(b[i]) < 1e30f) bm = fmaxf(bm, fabsf(b[i]));
  }
  bm = lanes_max<LPT>(bm);

  for (int r0 = wv * TPW; r0 < ntok; r0 += 4 * TPW) {
    const int local = r0 + sub;
    const int64_t t = t0 + min(local, ntok - 1);
    const bool active = local < ntok && (!mask || mask[t] != 0);
    const float* row = logits + t * p.E;
    float x[EPL], c[EPL];
    if (vec) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4) {
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (active && i < n) v = *(const float4*)(row + base + i);
        x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) x[i] = active && i < n ? row[base + i] : -INFINITY;
    }
    float top = 0.0f, sum = 1.0f, inv = 1.0f;
    if constexpr (!SIG) {
      top = x[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) top = fmaxf(top, x[i]);
      top = lanes_max<LPT>(top);
      if (top == -INFINITY) top = 0.0f;
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) sum += c[i] = __expf(x[i] - top);
      sum = lanes_sum<LPT>(sum);
      inv = 1.0f / sum;
    }
    bool odd = false;  // something for the 64-bit path
    float b1 = kNone, b2 = kNone;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float s = SIG ? __builtin_amdgcn_rcpf(1.0f + __expf(-x[i])) : c[i] * inv;
      const float v = s + b[i];
      const bool barred = x[i] == -INFINITY || b[i] == -INFINITY;
      odd |= !barred && !(fabsf(v) < 1e30f);
      c[i] = barred ? kNone : __uint_as_float((__float_as_uint(v) & ~15u) | (15 - i));
      b2 = __builtin_amdgcn_fmed3f(b1, b2, c[i]);
      b1 = fmaxf(b1, c[i]);
    }
    constexpr float kOff = SIG ? 0x1p-18f : 0x1p-16f;
    auto apart = [&](float hi, float lo) __attribute__((always_inline)) { return hi - lo > kOff * (fabsf(lo) + bm); };
    bool dropped = false;
    if (p.groups > 1) {
      float g1 = b1, g2 = b2;
      if (lg >= 2) merge_best<1>(g1, g2);
      if (lg >= 4) merge_best<2>(g1, g2);
      if (lg >= 8) merge_best<4>(g1, g2);
      if (LPT == 64 && lg >= 16) merge_best<8>(g1, g2);
      if (LPT == 64 && lg >= 32) merge_best<16>(g1, g2);
      const bool alive = g1 > -1e38f;
      const float v = p.group_best == 2 && g2 > -1e38f ? g1 + g2 : g1;
      int rank = 0;
      if constexpr (LPT == 16) {
        rank_by_rotation<1>(v, grp, lg, rank);
        rank /= lg;
      } else {
        for (int g = 0; g < p.groups; ++g) {
          const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), g * lg));
          rank += o > v || (o == v && g < grp);
        }
      }
      dropped = !alive || rank >= p.group_topk;
      const float least = -lanes_max<LPT>(dropped ? kNone : -v), next = lanes_max<LPT>(dropped && alive ? v : kNone);
      odd |= next > -1e38f && !(least - next > 2 * kOff * (fabsf(next) + 2 * bm));
      if (dropped) b1 = b2 = kNone;
    }
    if (!active) b1 = kNone - 1e35f * l;  // one winner in every round, which takes nothing
    bool half = false;                    // b2 has moved up
    float before = INFINITY;
    for (int j = 0; j <= p.k; ++j) {
      const float m = lanes_max<LPT>(b1);
      const bool win = b1 == m;
      odd |= __popcll(__ballot(win)) != TPW || (active && !apart(before, m));
      before = m;
      if (j == p.k) break;
      odd |= active && !(fabsf(m) > 1e-30f && m > -1e38f);
      const bool take = win && active;
      if (take) sh_ids[local * p.k + j] = base + 15 - (int)(__float_as_uint(m) & 15u);
      const bool refill = take && half;
      if (take) {
        b1 = b2;
        b2 = kNone;
        half = true;
      }
      if (__ballot(refill)) {
        float n1 = kNone, n2 = kNone;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const float v = c[i] < m && !dropped ? c[i] : kNone;
          n2 = __builtin_amdgcn_fmed3f(n1, n2, v);
          n1 = fmaxf(n1, v);
        }
        if (refill) {
          b1 = n1;
          b2 = n2;
          half = false;
        }
      }
    }
    // slot l of the lanes' token, and its weight
    const bool slot = l < p.k && local < ntok;
    int id = -1;
    float q = 0.0f;
    if (slot && active) id = min(sh_ids[local * p.k + l], p.E - 1);  // (past it: no expert was left, done again below)
    const float x1 = id >= 0 ? row[id] : 0.0f;
    float z;
    if constexpr (SIG) {
      const float m = p.renorm ? lanes_max<LPT>(id >= 0 ? fminf(x1, 0.0f) : -INFINITY) : 0.0f;
      z = id >= 0 ? expf(fminf(x1, 0.0f) - m) / (1.0f + expf(-fabsf(x1))) : 0.0f;
      if (p.renorm) z /= lanes_sum<LPT>(z);
    } else {
      const float m = p.renorm ? lanes_max<LPT>(id >= 0 ? x1 : -INFINITY) : top;
      z = id >= 0 ? expf(x1 - m) : 0.0f;
      z /= p.renorm ? lanes_sum<LPT>(z) : sum;
    }
    q = active ? z * p.scale : 0.0f;
    // tokens that are done again
    uint64_t again = __ballot(odd && active);
    while (again) {
      const int r = __builtin_ctzll(again) / LPT;
      again &= LPT == 64 ? 0 : ~(0xFFFFull << (16 * r));
      const Slot s = score_choose_token<EPL64>(p, logits + (t0 + r0 + r) * p.E, bias, sh_c[wv]);
      const int sid = LPT == 64 ? s.id : __shfl(s.id, l, 64);
      const float sw = LPT == 64 ? s.w : __shfl(s.w, l, 64);
      if (sub == r) {
        id = sid;
        q = sw;
      }
    }
    if (slot) {
      ids[t * p.k + l] = id;
      w[t * p.k + l] = q;
      sh_ids[local * p.k + l] = id;
    }
  }
  if (!segcnt && !perm) return;  // the plan is made elsewhere

  // ------------------------------------------------------------------ ranks and counts
  const int pairs = ntok * p.k, quarter = ((pairs + 3) / 4 + 63) / 64 * 64;
  const int lo = min(wv * quarter, pairs), hi = min(lo + quarter, pairs);
  int* run = sh_cnt + wv * p.E;
  for (int e = threadIdx.x; e < 4 * p.E; e += 256) sh_cnt[e] = 0;
  __syncthreads();
  for (int i = lo + lane; i < hi; i += 64)
    if (sh_ids[i] >= 0) atomicAdd(&run[sh_ids[i]], 1);
  __syncthreads();
  int* start = (int*)sh_c;  // first positions of the experts, where the block is the whole batch
  for (int e = threadIdx.x; e < p.E; e += 256) {
    int at = 0;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int c = sh_cnt[v * p.E + e];
      sh_cnt[v * p.E + e] = at;
      at += c;
    }
    if (perm) start[e] = at;
    else segcnt[(int64_t)blockIdx.x * p.E + e] = at;
  }
  __syncthreads();
  if (perm) {  // counts, and their exclusive sum by one wave
    if (wv == 0) {
      int before = 0;
      for (int e0 = 0; e0 < p.E; e0 += 64) {
        const int e = e0 + lane, c = e < p.E ? start[e] : 0;
        int x = c;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int y = __shfl_up(x, o, 64);
          if (lane >= o) x += y;
        }
        if (e < p.E) {
          counts[e] = c;
          offsets[e] = start[e] = before + x - c;
        }
        before += __shfl(x, 63, 64);
      }
      if (lane == 0) offsets[p.E] = before;
    }
    __syncthreads();
  }
  int bits = 1;
  while ((1 << bits) < p.E) ++bits;
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  for (int i0 = lo; i0 < hi; i0 += 64) {
    const int i = i0 + lane;
    const int e = i < hi ? sh_ids[i] : -1;
    uint64_t same = __ballot(e >= 0);
    for (int x = 0; x < bits; ++x) {
      const uint64_t set = __ballot((e >> x) & 1);
      same &= (e >> x) & 1 ? set : ~set;
    }
    int rank = 0;
    if (e >= 0) rank = run[e] + __popcll(same & below);
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && (same & below) == 0) run[e] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (i < hi) {
      if (!perm) {
        ranks[t0 * p.k + i] = (uint16_t)rank;
      } else if (e >= 0) {
        perm[start[e] + rank] = i;
        inv_perm[i] = start[e] + rank;
      } else {
        inv_perm[i] = -1;
      }
    }
  }
}

// Each expert's counts over the blocks: exclusive sums in their place, the total in counts.  64 experts a
// block, a sixteenth of the rows a wave.
__global__ __launch_bounds__(1024) void score_scan_kernel(int32_t* __restrict__ segcnt, int E, int S,
                                                          int32_t* __restrict__ counts) {
  __shared__ int part[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, e = blockIdx.x * 64 + lane;
  constexpr int ROWS = kSegments / 16;
  const int per = (S + 15) / 16, lo = wv * per;
  int v[ROWS], sum = 0;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    v[i] = i < per && lo + i < S && e < E ? segcnt[(int64_t)(lo + i) * E + e] : 0;
    sum += v[i];
  }
  part[wv][lane] = sum;
  __syncthreads();
  int at = 0, total = 0;
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    if (x < wv) at += part[x][lane];
    total += part[x][lane];
  }
  if (e >= E) return;
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    if (i < per && lo + i < S) {
      segcnt[(int64_t)(lo + i) * E + e] = at;
      at += v[i];
    }
  if (wv == 0) counts[e] = total;
}

// Positions of the pairs: the expert's first, its pairs in the blocks before, the rank in the block.
__global__ __launch_bounds__(256) void score_place_kernel(const int32_t* __restrict__ ids, int64_t pairs, int E, int seg_pairs,
                                                          const int32_t* __restrict__ segbase,
                                                          const uint16_t* __restrict__ ranks,
                                                          const int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                          int32_t* __restrict__ perm, int32_t* __restrict__ inv_perm) {
  __shared__ int start[1024], part[4];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int e0 = threadIdx.x * 4;
  int c[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) sum += c[i] = e0 + i < E ? counts[e0 + i] : 0;
  int x = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  if (lane == 63) part[wv] = x;
  __syncthreads();
  int at = x - sum;
  for (int i = 0; i < wv; ++i) at += part[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (e0 + i < E) {
      start[e0 + i] = at;
      if (blockIdx.x == 0) offsets[e0 + i] = at;
    }
    at += c[i];
  }
  if (blockIdx.x == 0 && threadIdx.x == 255) offsets[E] = at;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t q = (int64_t)blockIdx.x * 1024 + 256 * i + threadIdx.x;
    if (q >= pairs) return;
    const int e = ids[q];
    int pos = -1;
    if (e >= 0) {
      pos = start[e] + segbase[q / seg_pairs * E + e] + ranks[q];
      perm[pos] = (int32_t)q;
    }
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
  const size_t lds = 4 * (size_t)p.E * sizeof(int);
  int32_t* perm = sp.S == 1 && o.perm ? o.perm : nullptr;
  const unsigned grid = (unsigned)sp.S;
  if (p.sigmoid)
    score_choose_fast_kernel<LPT, EPL, EPL64, true><<<grid, 256, lds, st>>>(p, logits, bias, mask, o.ids, o.w, sp.seg, segcnt,
                                                                           ranks, o.counts, o.offsets, perm, o.inv_perm);
  else
    score_choose_fast_kernel<LPT, EPL, EPL64, false><<<grid, 256, lds, st>>>(p, logits, bias, mask, o.ids, o.w, sp.seg, segcnt,
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
    if (!here) sp = SegPlan{kSegPairs / p.k, (int)((p.T + kSegPairs / p.k - 1) / (kSegPairs / p.k))};
    int32_t* segcnt = here && sp.S > 1 ? (int32_t*)ws : nullptr;
    uint16_t* ranks = (uint16_t*)(segcnt ? segcnt + (size_t)sp.S * p.E : nullptr);
    const RouteOut o{ids, w, counts, offsets, here ? perm : nullptr, inv_perm};
    const int n16 = lane_share(p, 16);
    if (n16 <= 4) launch_fast<16, 4, 1>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    else if (n16 <= 8) launch_fast<16, 8, 2>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    else if (n16 <= 16) launch_fast<16, 16, 4>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    else if (lane_share(p, 64) <= 8) launch_fast<64, 8, 8>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    else launch_fast<64, 16, 16>(p, logits, bias, mask, o, sp, segcnt, ranks, st);
    if (segcnt) {
      score_scan_kernel<<<(p.E + 63) / 64, 1024, 0, st>>>(segcnt, p.E, sp.S, counts);
      score_place_kernel<<<(unsigned)((pairs + 1023) / 1024), 256, 0, st>>>(ids, pairs, p.E, sp.seg * p.k, segcnt, ranks,
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
