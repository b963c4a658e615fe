// Load-balancing loss of the gate: balance loss, z-loss, per-expert counts, and their gradient.
//
// With l = logits, a token counts if its mask is set, it lies in a group (a run of tokens: a
// sequence, or the whole batch) and it has a logit that is not -inf (a NaN counts):
//   lse_t = log sum_e exp(l_te)        p_te = exp(l_te - lse_t)
//   c_ge  = routed slots of g's counted tokens at expert e,   P_ge = sum of their p_te,   N_g
//   balance = 1/G sum_{N_g > 0} E / (k N_g^2) sum_e c_ge P_ge      z = 1/N sum_t lse_t^2
//   dl_te = p_te [ a E/(k N_g^2 G) (c_ge - sum_i c_gi p_ti) + 2 b lse_t / N ],  counts constant.
// A router that scores the experts and keeps the top K: page "Az NVIDIA szerint tízszer gyorsabb
// lett a dropless MoE tanítása JAX-ban", section "A dropless MoE minden tokent feldolgoz"; uneven
// loads slow training: section "Az egyenetlen terhelés lassítja a tanítást".
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kBalThreads = 256;
constexpr int kBalRedThreads = 1024;

// Tokens of a tile: at most 1024 tiles, whose partial sums few blocks add, until a tile has 512 tokens (its
// fp32 sums stay short); then up to 65536 tiles.  Both directions of 131071 tokens, 256 experts in 37
// groups: with 512 tiles 5 % more, with 2048 tiles 3 %.  Short batches: one tile, and so one launch, up
// to 128 tokens (100 x 128 as two tiles: 25 % more); then tiles of 32 tokens up to 8192 (5000 x 119 by 64:
// 3 % more), of 64 behind (16384 x 128 by 128: 6 % more).  Measured at 119 to 256 experts; the number of
// experts is not looked at.  What the kernels take by this rule stands at each of them.
int balance_tile(int64_t T) {
  if (T <= 128) return 128;
  int64_t t = (T + 1023) / 1024;
  if (t > 512) t = 512;
  if (t < (T + 65535) / 65536) t = (T + 65535) / 65536;
  const int least = T <= 8192 ? 32 : 64;
  return t < least ? least : (int)t;
}

int64_t al256i(int64_t x) { return (x + 255) & ~(int64_t)255; }

struct BalWs {
  float* P;        // [slots][E] partial sums of p
  int32_t* C;      // [slots][E] partial counts
  int32_t* n;      // [slots] counted tokens
  float* z;        // [slots] sum of lse^2
  double* part;    // [S][chunks] balance terms
  double* zpart;   // [S]
  int64_t bytes;
};

BalWs bal_ws(int64_t T, int64_t E, int64_t S, char* ws) {
  const int64_t tiles = T > 0 ? (T + balance_tile(T) - 1) / balance_tile(T) : 0;
  const int64_t slots = tiles + S, chunks = (E + 63) / 64;
  BalWs w{};
  int64_t off = 0;
  w.P = (float*)(ws + off);
  off += al256i(slots * E * 4);
  w.C = (int32_t*)(ws + off);
  off += al256i(slots * E * 4);
  w.n = (int32_t*)(ws + off);
  off += al256i(slots * 4);
  w.z = (float*)(ws + off);
  off += al256i(slots * 4);
  w.part = (double*)(ws + off);
  off += al256i(S * chunks * 8);
  w.zpart = (double*)(ws + off);
  off += al256i(S * 8);
  w.bytes = off;
  return w;
}

// Columns of 64 a block of the reduction takes: all of them while its 16 waves then read few rows each
// (one block, and no launch for the losses, if there is one group), else one.  16384 x 128 (2 x 257 rows):
// by two blocks 0.9 us more; 8192 x 256 (4 x 257): by one block 2.2 us more.
int balance_wide(int64_t T, int64_t E, int64_t S) {
  const int64_t rows = T > 0 ? (T + balance_tile(T) - 1) / balance_tile(T) / S + 1 : 1;
  int w = 1;
  while (w * 64 < E) w *= 2;
  return rows * w <= 600 ? w : 1;
}

// Last group whose first token is at or before t (-1: none).
__device__ __forceinline__ int group_of(const int32_t* off, int S, int t) {
  int lo = 0, hi = S + 1;  // off[0..S]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid + 1; else hi = mid;
  }
  return lo - 1;
}

// The same for a whole wave: a few offsets a lane, all loaded at once, where few loads cover them.
__device__ __forceinline__ int wave_group_of(const int32_t* off, int S, int t) {
  if (S >= 256) return group_of(off, S, t);
  const int lane = threadIdx.x & 63;
  int n = -1;
#pragma unroll
  for (int q = 0; q < 256; q += 64)
    if (q <= S) n += __popcll(__ballot(q + lane <= S && off[q + lane <= S ? q + lane : 0] <= t));
  return n;
}

constexpr int kL = 16;                      // lanes a token: a DPP row, so its sums need no LDS
constexpr int kRows = kBalThreads / kL;     // tokens a block takes at a time

// A row of E values over kL lanes: lane l holds the columns (n*kL + l)*V + v.
template <int V, int N>
__device__ __forceinline__ void load_row(const float* row, int E, int l, float fill, float (&x)[V * N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * kL + l) * V;
    if (V == 4) {
      float4 q = make_float4(fill, fill, fill, fill);
      if (c < E) q = *(const float4*)(row + c);
      x[n * V] = q.x, x[n * V + 1] = q.y, x[n * V + 2] = q.z, x[n * V + 3] = q.w;
    } else {
      x[n] = c < E ? row[c] : fill;
    }
  }
}

// Where a tile that is the whole batch, one group, puts its results (counts NULL: it is not)
struct BalOut {
  int32_t* counts;
  int32_t* tokens;
  float* losses;
};

// The losses of a batch that one block has seen whole.
template <int kCols>
__device__ __forceinline__ void whole_losses(const float (&shP)[4][kCols], const int32_t (&hist)[kCols],
                                             const int32_t (&sh_n)[4], const float (&sh_z)[4], int E, int k,
                                             const BalOut& o) {
  __shared__ double sh[4];
  double dot = 0.0;
  for (int c = threadIdx.x; c < E; c += kBalThreads) {
    o.counts[c] = hist[c];
    dot += (double)((shP[0][c] + shP[1][c]) + (shP[2][c] + shP[3][c])) * (double)hist[c];
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) dot += __shfl_xor(dot, m, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = dot;
  __syncthreads();
  if (threadIdx.x != 0) return;
  const int32_t n = sh_n[0] + sh_n[1] + sh_n[2] + sh_n[3];
  dot = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  const double z = ((double)sh_z[0] + (double)sh_z[1]) + ((double)sh_z[2] + (double)sh_z[3]);
  o.losses[0] = n > 0 ? (float)(dot * (double)E / ((double)k * (double)n * (double)n)) : 0.0f;
  o.losses[1] = n > 0 ? (float)(z / n) : 0.0f;
  o.tokens[0] = o.tokens[1] = n;
  o.tokens[2] = n > 0;
}

}  // namespace

// One block per tile of consecutive tokens, kL lanes per token, U tokens of a lane group in flight;
// each lane keeps the sums of p of its own columns.  A tile is cut where a group ends; the piece of
// tile b in group g has the slot b + g, which no other piece has (both grow along the tokens).  Where
// tiles are few, a tile's pieces are shared by blocks (gridDim.y of them: 42 tokens of 385 in 43 groups
// 6 us, by one block 83 us more).
// 131071 x 256, in one group and in 37: 31 us, 4.5 TB/s of logits and slots, bound by the loads that four
// waves a SIMD keep in flight around each token's two dependent sums (a whole wave for each token, with
// shuffles through LDS: 86 us more; four tokens in flight: 2 % less in one group, 7 % more in 37).  More
// experts leave three and two waves a SIMD and one token in flight: 65536 x 384 28 us, 65536 x 512 33,
// 32768 x 1024 31 (3.6, 4.1 and 4.4 TB/s).  16384 x 128: 7 us, of which the memory needs 1.4.
template <int V, int N>
__global__ __launch_bounds__(kBalThreads) void balance_stats_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ goff, int T, int E, int k, int S, int tile, float* __restrict__ lse_out,
    float* __restrict__ Pp, int32_t* __restrict__ Cp, int32_t* __restrict__ np, float* __restrict__ zp, BalOut whole) {
  constexpr int kCols = V * N * kL;
  constexpr int U = V * N <= 16 ? 2 : 1;
  __shared__ float shP[4][kCols];
  __shared__ int32_t hist[kCols];
  __shared__ int32_t sh_n[4];
  __shared__ float sh_z[4];
  const int tid = threadIdx.x, wv = tid >> 6, l = tid % kL, r = tid / kL;
  const int t0 = blockIdx.x * tile, t1 = T - t0 < tile ? T : t0 + tile;
  // the pieces of the tile: its part of each group, of the tokens before the first (-1) and behind the last
  for (int g = (goff ? wave_group_of(goff, S, t0) : 0) + blockIdx.y; g <= S; g += gridDim.y) {
    int a = t0, z = t1;
    if (goff) {
      if (g >= 0 && goff[g] > a) a = goff[g];
      if (a >= t1) break;
      if (g < S && goff[g + 1] < z) z = goff[g + 1];
      if (z <= a) continue;  // an empty group
    } else if (g > 0) {
      break;
    }
    const bool in = g >= 0 && g < S;
    for (int c = tid; c < kCols; c += kBalThreads) hist[c] = 0;
    __syncthreads();
    float acc[V * N];
#pragma unroll
    for (int i = 0; i < V * N; ++i) acc[i] = 0.0f;
    float zs = 0.0f;
    int cnt = 0;
    for (int64_t tb = a + r; tb < z; tb += kRows * U) {
      float x[U][V * N];
      int first[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {  // every load before the first use
        const int64_t t = tb + u * kRows;
        on[u] = t < z && in && (!mask || mask[t] != 0);
        first[u] = -1;
        if (on[u]) {
          load_row<V, N>(logits + t * E, E, l, -INFINITY, x[u]);
          if (l < k) first[u] = ids[t * k + l];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = tb + u * kRows;
        if (t >= z) break;
        float lse = -INFINITY;
        if (on[u]) {
          float mx = x[u][0];
#pragma unroll
          for (int i = 1; i < V * N; ++i) mx = fmaxf(mx, x[u][i]);
          mx = row16_max(mx);
          if (mx == -INFINITY) {
            // a maximum drops NaN beside -inf (another expert's, or behind the row): a token has no choice only
            // if all its logits are -inf
            bool other = false;
#pragma unroll
            for (int i = 0; i < V * N; ++i) other |= x[u][i] != -INFINITY;
            if (__ballot(other) >> (tid & 48) & 0xffff) mx = NAN;
          }
          if (mx != -INFINITY) {  // the same for the token's lanes
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < V * N; ++i) {
              x[u][i] = __expf(x[u][i] - mx);
              s += x[u][i];
            }
            s = row16_sum(s);
            const float inv = 1.0f / s;
#pragma unroll
            for (int i = 0; i < V * N; ++i) acc[i] += x[u][i] * inv;
            lse = mx + logf(s);
            zs += lse * lse;
            ++cnt;
            if (first[u] >= 0 && first[u] < E) atomicAdd(&hist[first[u]], 1);  // integers: any order gives the same
            for (int j = l + kL; j < k; j += kL) {
              const int e = ids[t * k + j];
              if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
            }
          }
        }
        if (l == 0) lse_out[t] = lse;
      }
    }
    if (in) {
      // the rows of a wave, then the four waves, in fixed order
#pragma unroll
      for (int m = kL; m < 64; m <<= 1) {
#pragma unroll
        for (int i = 0; i < V * N; ++i) acc[i] += __shfl_xor(acc[i], m, 64);
        zs += __shfl_xor(zs, m, 64);
        cnt += __shfl_xor(cnt, m, 64);
      }
      if ((tid & 63) < kL) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int v = 0; v < V; ++v) shP[wv][(n * kL + l) * V + v] = acc[n * V + v];
        if (l == 0) sh_n[wv] = cnt, sh_z[wv] = zs;
      }
      __syncthreads();
      if (whole.counts) {
        whole_losses(shP, hist, sh_n, sh_z, E, k, whole);
        return;
      }
      const int64_t slot = (int64_t)blockIdx.x + g;
      for (int c = tid; c < E; c += kBalThreads) {
        Pp[slot * E + c] = (shP[0][c] + shP[1][c]) + (shP[2][c] + shP[3][c]);
        Cp[slot * E + c] = hist[c];
      }
      if (tid == 0) {
        np[slot] = sh_n[0] + sh_n[1] + sh_n[2] + sh_n[3];
        zp[slot] = (sh_z[0] + sh_z[1]) + (sh_z[2] + sh_z[3]);
      }
    }
    __syncthreads();
  }
}

// One block per (chunk of 64 * W columns, group): its 16 waves are W columns of 64 by 16 / W rows; adds
// the pieces of the group's tiles in a fixed order (64-bit sums) and writes the counts.  A grid of one
// block writes the losses too; else balance_final_kernel does (a last block found by a counter needs a
// fence that writes the L2s back: 14 us for 2 blocks, against 4 and 4 for the two launches or 6 for one
// block).  Latency: 16384 x 128, 256 pieces: 6 us; 131071 x 256, 37 groups: 7 us and 4.
template <int W>
__global__ __launch_bounds__(kBalRedThreads) void balance_reduce_kernel(
    const float* __restrict__ Pp, const int32_t* __restrict__ Cp, const int32_t* __restrict__ np,
    const float* __restrict__ zp, const int32_t* __restrict__ goff, int T, int E, int k, int S, int tile,
    int32_t* __restrict__ counts, int32_t* __restrict__ tokens, float* __restrict__ losses, double* part,
    double* zpart) {
  constexpr int kW = kBalRedThreads / 64, kR = kW / W;
  __shared__ double shP[kW][64];
  __shared__ int32_t shC[kW][64];
  __shared__ int32_t sh_n[kW];
  __shared__ double sh_z[kW];
  __shared__ double sh[64];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, row = wv / W;
  const int g = blockIdx.y, c = (blockIdx.x * W + wv % W) * 64 + lane, chunks = gridDim.x;
  int a = 0, z = T;
  if (goff) {
    a = goff[g] < 0 ? 0 : goff[g];
    z = goff[g + 1] > T ? T : goff[g + 1];
  }
  const int b0 = z > a ? a / tile : 0, b1 = z > a ? (z - 1) / tile + 1 : 0;
  int32_t n = 0;
  double zs = 0.0;
  for (int b = b0 + tid; b < b1; b += kBalRedThreads) {
    n += np[b + g];
    zs += (double)zp[b + g];
  }
  double P = 0.0;
  int32_t C = 0;
  if (c < E) {
#pragma unroll 8
    for (int b = b0 + row; b < b1; b += kR) {
      const int64_t at = ((int64_t)b + g) * E + c;
      P += (double)Pp[at];
      C += Cp[at];
    }
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    n += __shfl_xor(n, m, 64);
    zs += __shfl_xor(zs, m, 64);
  }
  shP[wv][lane] = P;
  shC[wv][lane] = C;
  if (lane == 0) sh_n[wv] = n, sh_z[wv] = zs;
  __syncthreads();
  n = 0;
  zs = 0.0;
#pragma unroll
  for (int w = 0; w < kW; ++w) n += sh_n[w], zs += sh_z[w];
  double dot = 0.0;
  if (row == 0) {
#pragma unroll
    for (int q = 1; q < kR; ++q) P += shP[q * W + wv][lane], C += shC[q * W + wv][lane];
    if (c < E) {
      counts[(int64_t)g * E + c] = C;
      dot = (double)C * P;
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) dot += __shfl_xor(dot, m, 64);
    if (lane == 0) sh[wv] = dot;
  }
  __syncthreads();
  if (tid != 0) return;
  dot = 0.0;
#pragma unroll
  for (int w = 0; w < W; ++w) dot += sh[w];
  const double term = n > 0 ? dot * (double)E / ((double)k * (double)n * (double)n) : 0.0;
  if (gridDim.x * gridDim.y == 1) {  // one group, seen whole
    losses[0] = (float)term;
    losses[1] = n > 0 ? (float)(zs / n) : 0.0f;
    tokens[0] = tokens[1] = n;
    tokens[2] = n > 0;
    return;
  }
  part[(int64_t)g * chunks + blockIdx.x] = term;
  if (blockIdx.x == 0) tokens[g] = n, zpart[g] = zs;
}

// The losses from the groups' terms, in a fixed order, by one wave for few of them.
template <int NT>
__global__ __launch_bounds__(NT) void balance_final_kernel(const double* part, const double* zpart, int S,
                                                                       int chunks, int32_t* tokens, float* losses) {
  __shared__ double sh[4][NT / 64];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  double bal = 0.0, zs = 0.0;
  int32_t groups = 0, total = 0;
  for (int64_t i = tid; i < (int64_t)S * chunks; i += NT) bal += part[i];
  for (int i = tid; i < S; i += NT) {
    const int32_t m = tokens[i];
    total += m;
    groups += m > 0;
    zs += zpart[i];
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    bal += __shfl_xor(bal, m, 64);
    zs += __shfl_xor(zs, m, 64);
    total += __shfl_xor(total, m, 64);
    groups += __shfl_xor(groups, m, 64);
  }
  if (lane == 0) sh[0][wv] = bal, sh[1][wv] = zs, sh[2][wv] = total, sh[3][wv] = groups;
  __syncthreads();
  if (tid != 0) return;
  bal = 0.0, zs = 0.0;
  double n = 0.0, g = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) bal += sh[0][w], zs += sh[1][w], n += sh[2][w], g += sh[3][w];
  losses[0] = g > 0.0 ? (float)(bal / g) : 0.0f;
  losses[1] = n > 0.0 ? (float)(zs / n) : 0.0f;
  tokens[S] = (int32_t)n;
  tokens[S + 1] = (int32_t)g;
}

// The gradient: kL lanes per token.  Since sum_e p = 1, an integer near their mean is taken off the
// counts first, which loses nothing and keeps the difference from cancelling.  Bound by HBM: 131071 x 256
// in 37 groups with another gradient added: 69 us, 5.8 TB/s; written past the caches (cached stores: 5 us
// more).  16384 x 128: 7 us.
template <int V, int N>
__global__ __launch_bounds__(kBalThreads) void balance_grad_kernel(
    const float* __restrict__ logits, const float* __restrict__ lse_in, const int32_t* __restrict__ goff,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens, const float* __restrict__ d_losses, int T,
    int E, int k, int S, int tile, const float* d_in, float* d_out) {
  const int tid = threadIdx.x, l = tid % kL, r = tid / kL;
  const int t0 = blockIdx.x * tile, t1 = T - t0 < tile ? T : t0 + tile;
  const int g0 = goff ? wave_group_of(goff, S, t0) : 0, end0 = goff ? (g0 < S ? goff[g0 + 1] : t1) : T;
  int lo = 0, hi = -1;  // the group's tokens: no group yet
  float c[V * N];
#pragma unroll
  for (int i = 0; i < V * N; ++i) c[i] = 0.0f;
  float ca = 0.0f;
  const int32_t total = tokens[S];
  const float cb = total > 0 ? 2.0f * d_losses[1] / (float)total : 0.0f;
  for (int64_t t = t0 + r; t < t1; t += kRows) {
    const int64_t row = t * E;
    const float lse = lse_in[t];
    float p[V * N], d[V * N];
    load_row<V, N>(logits + row, E, l, -INFINITY, p);
    if (d_in) {
      load_row<V, N>(d_in + row, E, l, 0.0f, d);
    } else {
#pragma unroll
      for (int i = 0; i < V * N; ++i) d[i] = 0.0f;
    }
    if (lse != -INFINITY) {  // else what was read of the logits is not used
      if (t < lo || t >= hi) {
        int g = t < end0 ? g0 : group_of(goff, S, (int)t);
        g = g < 0 ? 0 : (g >= S ? S - 1 : g);  // a counted token lies in a group
        lo = goff ? goff[g] : 0;
        hi = goff ? goff[g + 1] : T;
        const int32_t n = tokens[g];
        const int32_t mean = (int32_t)((int64_t)k * n / E);
        const int32_t* cg = counts + (int64_t)g * E;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int col = (i * kL + l) * V + v;
            c[i * V + v] = col < E ? (float)(cg[col] - mean) : 0.0f;
          }
        ca = n > 0 ? (float)((double)d_losses[0] * (double)E / ((double)k * n * (double)n * (double)tokens[S + 1])) : 0.0f;
      }
      // p = e / sum e: lse is rounded to its own size, and exp(l - lse) alone would be off by as much (of logits
      // past 2^27 the log E is lost: by a factor of E).  One sum more: 16384 x 128 0.2 us
      float dot = 0.0f, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V * N; ++i) {
        p[i] = __expf(p[i] - lse);
        sum += p[i];
        dot += c[i] * p[i];
      }
      const float inv = __builtin_amdgcn_rcpf(row16_sum(sum));  // 1 ulp; the sum is 1 but for lse's rounding
      dot = row16_sum(dot) * inv;
      const float cn = ca * inv, zc = cb * lse * inv;
#pragma unroll
      for (int i = 0; i < V * N; ++i) d[i] += p[i] * (cn * (c[i] - dot) + zc);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int col = (n * kL + l) * V;
      if (col >= E) continue;
      if (V == 4)
        __builtin_nontemporal_store(f32x4_t{d[n * V], d[n * V + 1], d[n * V + 2], d[n * V + 3]},
                                    (f32x4_t*)(d_out + row + col));
      else
        d_out[row + col] = d[n];
    }
  }
}

namespace {

// The fewest columns a lane that hold a row; rows of a multiple of 4 columns are 16-byte aligned and
// move as vectors.
#define MOE_BAL_DISPATCH(E, CALL)                  \
  do {                                             \
    if ((E) % 4 == 0) {                            \
      if ((E) <= 64) { CALL(4, 1); }               \
      else if ((E) <= 128) { CALL(4, 2); }         \
      else if ((E) <= 256) { CALL(4, 4); }         \
      else if ((E) <= 512) { CALL(4, 8); }         \
      else { CALL(4, 16); }                        \
    } else {                                       \
      if ((E) <= 64) { CALL(1, 4); }               \
      else if ((E) <= 128) { CALL(1, 8); }         \
      else if ((E) <= 256) { CALL(1, 16); }        \
      else if ((E) <= 512) { CALL(1, 32); }        \
      else { CALL(1, 64); }                        \
    }                                              \
  } while (0)

}  // namespace

size_t balance_ws_bytes(int64_t T, int64_t E, int64_t S) { return (size_t)bal_ws(T, E, S, nullptr).bytes; }

hipError_t launch_balance_forward(const float* logits, const int32_t* ids, const uint8_t* mask, const int32_t* goff,
                                  int T, int E, int k, int S, int32_t* counts, int32_t* tokens, float* losses,
                                  float* lse, void* ws, hipStream_t st) {
  const BalWs w = bal_ws(T, E, S, (char*)ws);
  const int tile = balance_tile(T);
  const unsigned tiles = (unsigned)((T + (int64_t)tile - 1) / tile);
  // one tile and one group of all tokens: the one block writes the results
  const bool one = tiles == 1 && !goff;
  const BalOut whole{one ? counts : nullptr, tokens, losses};
  if (tiles > 0) {
    const dim3 grid(tiles, tiles >= 512 ? 1 : 512 / tiles < (unsigned)S ? 512 / tiles : S);
#define MOE_BAL_CALL(V, N)                                                                                       \
  balance_stats_kernel<V, N><<<grid, kBalThreads, 0, st>>>(logits, ids, mask, goff, T, E, k, S, tile, lse, w.P, \
                                                            w.C, w.n, w.z, whole)
    MOE_BAL_DISPATCH(E, MOE_BAL_CALL);
#undef MOE_BAL_CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || one) return e;
  }
  const int wide = balance_wide(T, E, S);
  const int chunks = (E + 64 * wide - 1) / (64 * wide);
  const dim3 grid(chunks, S);
#define MOE_BAL_CALL(W)                                                                                             \
  balance_reduce_kernel<W><<<grid, kBalRedThreads, 0, st>>>(w.P, w.C, w.n, w.z, goff, T, E, k, S, tile, counts, \
                                                            tokens, losses, w.part, w.zpart)
  if (wide == 1) MOE_BAL_CALL(1);
  else if (wide == 2) MOE_BAL_CALL(2);
  else if (wide == 4) MOE_BAL_CALL(4);
  else if (wide == 8) MOE_BAL_CALL(8);
  else MOE_BAL_CALL(16);
#undef MOE_BAL_CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks * S == 1) return e;
  if ((int64_t)chunks * S <= 512)
    balance_final_kernel<64><<<1, 64, 0, st>>>(w.part, w.zpart, S, chunks, tokens, losses);
  else
    balance_final_kernel<kBalRedThreads><<<1, kBalRedThreads, 0, st>>>(w.part, w.zpart, S, chunks, tokens, losses);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const float* logits, const float* lse, const int32_t* goff, const int32_t* counts,
                                   const int32_t* tokens, const float* d_losses, int T, int E, int k, int S,
                                   const float* d_in, float* d_out, hipStream_t st) {
  if (T == 0) return hipSuccess;
  // tokens of a block (128 experts: 2048 tokens by 32 0.5 us more; 8192 by 16 1.0 more, by 64 2.3; 32768 by
  // 32 1.6 more; 131071 x 256 by 32 4 more); a grid's threads fit 32 bits
  const int tile = T <= 4096 ? 16 : T <= 12288 ? 32 : T <= (1 << 27) ? 64 : 1024;
  const unsigned tiles = (unsigned)((T + (int64_t)tile - 1) / tile);
#define MOE_BAL_CALL(V, N)                                                                                       \
  balance_grad_kernel<V, N><<<tiles, kBalThreads, 0, st>>>(logits, lse, goff, counts, tokens, d_losses, T, E, k, \
                                                           S, tile, d_in, d_out)
  MOE_BAL_DISPATCH(E, MOE_BAL_CALL);
#undef MOE_BAL_CALL
  return hipGetLastError();
}

}  // namespace moe
