// Scored router: expert selection from gate logits, its backward, and the
// balance losses. The contract of each entry point is in include/moe.h.
//
// Scores s[t][e] are sigmoid(l) or softmax(l) over the E experts; the choice
// goes by the key c = s + balance_bias (the bias chooses, it does not weigh).
// Keys are compared as doubles: neighbouring scores of a 256-expert row are
// about 1/256 apart, so in fp32 (2^-24 per score) one row in some ten thousand
// would order two experts by rounding; in doubles the order is the formula's.
#include <type_traits>

#include "common.h"
#include "router.h"

namespace moe {

namespace {

constexpr float kF32Max = 3.402823466e38f;

// A logit as the scores see it: out of the choice when -inf or NaN; +inf counts
// as the largest finite value.
__device__ __forceinline__ bool live_value(float v) { return v > -INFINITY; }  // false for NaN

// Doubles as unsigned integers of the same order (c is never NaN; -0 as +0).
__device__ __forceinline__ uint64_t order_bits(double c) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(c + 0.0));
  return b ^ ((b >> 63) ? ~uint64_t(0) : (uint64_t(1) << 63));
}
constexpr uint64_t kKeyTaken = 0;  // below every key: chosen already, or no expert
constexpr uint64_t kKeyDead = 1;   // out of the choice: chosen last, in ascending order

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int off) {
  const uint32_t lo = __shfl_xor(static_cast<uint32_t>(v), off), hi = __shfl_xor(static_cast<uint32_t>(v >> 32), off);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

__device__ __forceinline__ float sigmoidf(float l) { return 1.0f / (1.0f + expf(-l)); }
// sigmoid(l) / exp(min(m, 0)) for l <= m: no underflow where all of a row's
// scores are tiny, since only ratios of them are used.
__device__ __forceinline__ float sigmoid_scaled(float l, float m) {
  return m >= 0.0f ? sigmoidf(l) : expf(l - m) / (1.0f + expf(l));
}

// lane's experts: lane * VPL + i, i < VPL (so lower lanes hold lower experts)
template <int VPL>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, float (&l)[VPL]) {
  const int e0 = (threadIdx.x & 63) * VPL;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float v = e0 + i < E ? row[e0 + i] : -INFINITY;
    l[i] = live_value(v) ? fminf(v, kF32Max) : -INFINITY;
  }
}

// One wave per token: scores and keys in registers, groups ranked from LDS,
// then k rounds of a wave arg-max over (key, logit, lower expert).
template <int VPL>
__global__ __launch_bounds__(64) void select_kernel(SelectOpts o, const float* __restrict__ logits,
                                                    const float* __restrict__ bias, int T, int E, int k,
                                                    int32_t* __restrict__ idx, float* __restrict__ w) {
  __shared__ uint64_t skey[64 * VPL];
  __shared__ float sel[64 * VPL];  // logits of the chosen experts (NaN: out of the choice)
  const int lane = threadIdx.x;
  const int e0 = lane * VPL;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
  __syncthreads();  // the previous token's LDS is read out
  float l[VPL];
  load_row<VPL>(logits + t * E, E, l);

  // scores and keys
  uint64_t key[VPL];
  float m = l[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
  m = wave_max(m);  // -inf when nothing is live
  double z[VPL], zs = 0.0;
  if (!o.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      z[i] = live_value(l[i]) ? exp(static_cast<double>(l[i]) - m) : 0.0;
      zs += z[i];
    }
    zs = wave_sum(zs);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float b = bias && e0 + i < E ? bias[e0 + i] : 0.0f;
    const bool live = live_value(l[i]) && live_value(b);
    double s = 0.0;
    if (live) s = o.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l[i]))) : z[i] / zs;
    key[i] = e0 + i >= E ? kKeyTaken : (live ? order_bits(s + b) : kKeyDead);
  }

  if (o.groups > 1) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) skey[e0 + i] = key[i];
    __syncthreads();
    const int per = E / o.groups;
    // lane g: group g's key, again as ordered bits (0: no live expert)
    uint64_t gk = 0;
    if (lane < o.groups) {
      uint64_t a = 0, b = 0;
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        const uint64_t v = skey[e];
        if (v > a) { b = a; a = v; }
        else if (v > b) b = v;
      }
      if (a > kKeyDead) {
        gk = a;
        if (o.top2 && b > kKeyDead) {
          const auto back = [](uint64_t q) {
            return __longlong_as_double(static_cast<long long>(q ^ ((q >> 63) ? (uint64_t(1) << 63) : ~uint64_t(0))));
          };
          gk = order_bits(back(a) + back(b));
        }
      }
    }
    int rank = 0;
    for (int g = 0; g < o.groups; ++g) {
      const uint64_t v = (static_cast<uint64_t>(__shfl(static_cast<uint32_t>(gk >> 32), g)) << 32) |
                         __shfl(static_cast<uint32_t>(gk), g);
      rank += v > gk || (v == gk && g < lane);
    }
    const uint64_t kept = __ballot(lane < o.groups && rank < o.topk_groups);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < E && !((kept >> ((e0 + i) / per)) & 1)) key[i] = kKeyDead;
  }

  for (int j = 0; j < k; ++j) {
    uint64_t bk = kKeyTaken;
    float bl = 0.0f;
    int be = E;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > bk || (key[i] == bk && key[i] > kKeyDead && l[i] > bl)) { bk = key[i]; bl = l[i]; be = e0 + i; }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const uint64_t ok = shfl_xor64(bk, off);
      const float ol = __shfl_xor(bl, off);
      const int oe = __shfl_xor(be, off);
      const bool tie = ok == bk;
      if (ok > bk || (tie && ok > kKeyDead && ol > bl) || (tie && (ok <= kKeyDead || ol == bl) && oe < be)) {
        bk = ok; bl = ol; be = oe;
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i == be) key[i] = kKeyTaken;
    if (lane == 0) {
      idx[t * k + j] = be;
      sel[j] = bk > kKeyDead ? bl : NAN;
    }
  }
  __syncthreads();

  // Weights in fp32 from the chosen logits; a renormalised weight is a ratio,
  // formed from scores scaled by the largest chosen one.
  float mx = -INFINITY;
  for (int j = lane; j < k; j += 64) mx = fmaxf(mx, live_value(sel[j]) ? sel[j] : -INFINITY);
  mx = wave_max(mx);
  const float inv_z = o.sigmoid ? 1.0f : static_cast<float>(1.0 / zs);
  auto score = [&](float v) {
    if (!live_value(v)) return 0.0f;
    if (o.renorm) return o.sigmoid ? sigmoid_scaled(v, mx) : expf(v - mx);
    return o.sigmoid ? sigmoidf(v) : expf(v - m) * inv_z;
  };
  float tot = 0.0f;
  if (o.renorm) {
    for (int j = lane; j < k; j += 64) tot += score(sel[j]);
    tot = wave_sum(tot);
  }
  const float f = o.renorm ? (tot > 0.0f ? o.scale / tot : 0.0f) : o.scale;
  for (int j = lane; j < k; j += 64) w[t * k + j] = score(sel[j]) * f;
  }
}

// Sequence bounds of row t: its start, length, id, and the number of sequences
// with rows. Offsets are clamped to [0, T] so that any values stay in bounds.
struct Seq {
  int id, len, filled, covered;
};
__device__ __forceinline__ int clamp_off(int32_t v, int T) { return v < 0 ? 0 : (v > T ? T : v); }
__device__ __forceinline__ Seq find_seq(const int32_t* __restrict__ off, int n_seq, int t, int T) {
  if (!off) return {0, T, T > 0, T};
  const int lane = threadIdx.x & 63;
  int id = 0, filled = 0;
  for (int s0 = 0; s0 < n_seq; s0 += 64) {
    const int s = s0 + lane;
    const bool in = s < n_seq;
    const int a = in ? clamp_off(off[s], T) : 0, b = in ? clamp_off(off[s + 1], T) : 0;
    id += __popcll(__ballot(in && b <= t));
    filled += __popcll(__ballot(in && b > a));
  }
  const int first = clamp_off(off[0], T), last = clamp_off(off[n_seq], T);
  if (t < first || t >= last || id >= n_seq) return {-1, 0, filled, last - first};
  return {id, clamp_off(off[id + 1], T) - clamp_off(off[id], T), filled, last - first};
}

// One wave per token. With w the selection's weights (zero for a slot whose
// expert was out of the choice), D = sum_j w_j dw_j:
//   renormalised:  dl[e_j] = w_j sum_i (w_i / scale)(dw_j - dw_i) (1 - s_j)   (sigmoid)
//                  the same without (1 - s_j)                     (softmax)
//   otherwise:     dl[e_j] = w_j dw_j (1 - s_j)                   (sigmoid)
//                  dl[e]   = [e = e_j] w_j dw_j - p_e D           (softmax, every e)
// and, with shares p~ (softmax: p; sigmoid: s over its row sum) and the balance
// loss's g_e = dB E f_e / (k n^2 filled), the z loss's lse = log sum exp l:
//   dl[e] += p~_e (g_e - sum p~ g) (1 - s_e if sigmoid) + dZ 2 lse p_e / covered.
template <int VPL>
__global__ __launch_bounds__(256) void select_backward_kernel(SelectOpts o, const float* __restrict__ logits,
                                                              const int32_t* __restrict__ idx,
                                                              const float* __restrict__ w,
                                                              const float* __restrict__ dw,
                                                              const float* __restrict__ dlosses,
                                                              const int32_t* __restrict__ load,
                                                              const int32_t* __restrict__ seq_offsets, int n_seq, int T,
                                                              int E, int k, float* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const int e0 = lane * VPL;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); t < T; t += 4 * static_cast<int64_t>(gridDim.x)) {
  const int64_t row = t * E;
  float l[VPL], dl[VPL], p[VPL];
  load_row<VPL>(logits + row, E, l);
  float m = l[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
  m = wave_max(m);
  float zs = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    p[i] = live_value(l[i]) ? expf(l[i] - m) : 0.0f;
    zs += p[i];
    dl[i] = 0.0f;
  }
  zs = wave_sum(zs);
  const float inv_z = zs > 0.0f ? 1.0f / zs : 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) p[i] *= inv_z;

  // the selection
  if (dw) {
    const int64_t a0 = t * k;
    float dsum = 0.0f;
    for (int j = lane; j < k; j += 64) {
      const float wj = o.sigmoid || o.renorm ? 0.0f : w[a0 + j];
      if (wj != 0.0f) dsum += wj * dw[a0 + j];  // a slot out of the choice adds nothing, whatever its dw
    }
    dsum = wave_sum(dsum);
    const float unit = o.renorm && o.scale != 0.0f ? 1.0f / o.scale : 0.0f;
    for (int j0 = 0; j0 < k; j0 += 64) {
      const int j = j0 + lane;
      int e = -1;
      float g = 0.0f;
      if (j < k) {
        e = idx[a0 + j];
        const float wj = w[a0 + j];
        if (wj != 0.0f) g = wj * dw[a0 + j];
        if (o.renorm) {
          // dw_j - sum_i v_i dw_i as sum_i v_i (dw_j - dw_i), v = w / scale summing to 1: nothing cancels
          g = 0.0f;
          for (int i = 0; i < k; ++i) {
            const float wi = w[a0 + i];  // the same for every lane
            if (wi != 0.0f && wj != 0.0f) g += wi * unit * (dw[a0 + j] - dw[a0 + i]);
          }
          g *= wj;
        }
      }
      const int n = min(64, k - j0);
      for (int q = 0; q < n; ++q) {
        const int eq = __builtin_amdgcn_readlane(e, q);
        const float gq = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), q));
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (e0 + i == eq) dl[i] += gq;
      }
    }
    if (o.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (dl[i] != 0.0f) dl[i] *= sigmoidf(-l[i]);
    } else if (!o.renorm) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) dl[i] -= p[i] * dsum;
    }
  }

  // the losses
  if (dlosses) {
    const Seq q = find_seq(seq_offsets, n_seq, static_cast<int>(t), T);
    if (q.id >= 0 && m > -INFINITY) {
      const float cb = static_cast<float>(static_cast<double>(dlosses[0]) * E /
                                          (static_cast<double>(k) * q.len * q.len * q.filled));
      float sh[VPL], tot = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        sh[i] = o.sigmoid ? (live_value(l[i]) ? sigmoid_scaled(l[i], m) : 0.0f) : p[i];
        tot += sh[i];
      }
      if (o.sigmoid) {
        tot = 1.0f / wave_sum(tot);
#pragma unroll
        for (int i = 0; i < VPL; ++i) sh[i] *= tot;
      }
      float g[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        g[i] = e0 + i < E ? cb * static_cast<float>(load[static_cast<int64_t>(q.id) * E + e0 + i]) : 0.0f;
        dot += sh[i] * g[i];
      }
      dot = wave_sum(dot);
      const float cz = dlosses[1] * 2.0f / static_cast<float>(q.covered) * (m + logf(zs));
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float v = sh[i] * (g[i] - dot);
        if (o.sigmoid && sh[i] != 0.0f) v *= sigmoidf(-l[i]);
        dl[i] += v + cz * p[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (e0 + i < E) dlogits[row + e0 + i] = dl[i];
  }
}

// ---------------------------------------------------------------- losses ----
// Part r of sequence s: its rows' shares p~ summed per expert (fp32 over at
// most a few dozen rows per wave; the parts are then summed in double), the
// loads counted (integers, any order gives the same), and sum lse^2 (double).
template <int VPL>
__global__ __launch_bounds__(256) void balance_part_kernel(SelectOpts o, const float* __restrict__ logits,
                                                           const int32_t* __restrict__ idx,
                                                           const int32_t* __restrict__ seq_offsets, int T, int E, int k,
                                                           float* __restrict__ part_p, int32_t* __restrict__ part_f,
                                                           double* __restrict__ part_z) {
  __shared__ int32_t cnt[64 * VPL];
  __shared__ float psum[4][64 * VPL];
  __shared__ double zsum[4];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r = blockIdx.x, s = blockIdx.y, parts = gridDim.x;
  const int a = seq_offsets ? clamp_off(seq_offsets[s], T) : 0, b = seq_offsets ? clamp_off(seq_offsets[s + 1], T) : T;
  const int64_t n = b > a ? b - a : 0;
  const int lo = a + static_cast<int>(n * r / parts), hi = a + static_cast<int>(n * (r + 1) / parts);
  for (int e = threadIdx.x; e < 64 * VPL; e += 256) cnt[e] = 0;
  __syncthreads();
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  double zacc = 0.0;
  for (int t = lo + wv; t < hi; t += 4) {
    float l[VPL], x[VPL];
    load_row<VPL>(logits + static_cast<int64_t>(t) * E, E, l);
    for (int j = lane; j < k; j += 64) {
      const int e = idx[static_cast<int64_t>(t) * k + j];
      if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
    if (m == -INFINITY) continue;
    float zs = 0.0f, tot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      x[i] = live_value(l[i]) ? expf(l[i] - m) : 0.0f;
      zs += x[i];
      if (o.sigmoid) {
        x[i] = live_value(l[i]) ? sigmoid_scaled(l[i], m) : 0.0f;
        tot += x[i];
      }
    }
    zs = wave_sum(zs);
    tot = 1.0f / (o.sigmoid ? wave_sum(tot) : zs);
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] += x[i] * tot;
    const double lse = static_cast<double>(m) + logf(zs);
    zacc += lse * lse;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) psum[wv][lane * VPL + i] = acc[i];
  if (lane == 0) zsum[wv] = zacc;
  __syncthreads();
  const int64_t base = (static_cast<int64_t>(s) * parts + r) * E;
  for (int e = threadIdx.x; e < E; e += 256) {
    part_p[base + e] = ((psum[0][e] + psum[1][e]) + psum[2][e]) + psum[3][e];
    part_f[base + e] = cnt[e];
  }
  if (threadIdx.x == 0) part_z[static_cast<int64_t>(s) * parts + r] = ((zsum[0] + zsum[1]) + zsum[2]) + zsum[3];
}

constexpr int kRedE = 16;  // experts per block of the part reduction

// Block (eb, s): parts summed in order for kRedE experts (16 slices of parts,
// then the slices in order), load[s][e] written, the experts' terms f * P added.
// term[s][eb]; block 0's slot [s][blocks] holds the sequence's sum of lse^2.
__global__ __launch_bounds__(256) void balance_reduce_kernel(const float* __restrict__ part_p,
                                                             const int32_t* __restrict__ part_f,
                                                             const double* __restrict__ part_z, int parts, int E,
                                                             double* __restrict__ term, int32_t* __restrict__ load) {
  __shared__ double sp[16][kRedE];
  __shared__ int32_t sf[16][kRedE];
  __shared__ double sz[256];
  const int s = blockIdx.y, el = threadIdx.x % kRedE, sl = threadIdx.x / kRedE;
  const int e = blockIdx.x * kRedE + el;
  double p = 0.0;
  int32_t f = 0;
  if (e < E)
    for (int r = sl; r < parts; r += 16) {
      const int64_t at = (static_cast<int64_t>(s) * parts + r) * E + e;
      p += part_p[at];
      f += part_f[at];
    }
  sp[sl][el] = p;
  sf[sl][el] = f;
  double z = 0.0;
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r < parts; r += 256) z += part_z[static_cast<int64_t>(s) * parts + r];
  sz[threadIdx.x] = z;
  __syncthreads();
  if (threadIdx.x < kRedE) {
    double ps = 0.0;
    int32_t fs = 0;
    for (int q = 0; q < 16; ++q) { ps += sp[q][threadIdx.x]; fs += sf[q][threadIdx.x]; }
    if (e < E) load[static_cast<int64_t>(s) * E + e] = fs;
    sp[0][threadIdx.x] = ps * fs;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int q = 0; q < kRedE; ++q) v += sp[0][q];
    double* row = term + static_cast<int64_t>(s) * (gridDim.x + 1);
    row[blockIdx.x] = v;
    if (blockIdx.x == 0) {
      double zt = 0.0;
      for (int q = 0; q < 256; ++q) zt += sz[q];
      row[gridDim.x] = zt;
    }
  }
}

// One wave: B = 1/filled sum_s E / (k n_s^2) sum_e f P, Z = sum lse^2 / covered.
__global__ __launch_bounds__(64) void balance_final_kernel(const double* __restrict__ term,
                                                           const int32_t* __restrict__ seq_offsets, int n_seq, int T,
                                                           int E, int k, int blocks, float* __restrict__ losses) {
  double bsum = 0.0, zsum = 0.0;
  int filled = 0, covered = 0;
  for (int s = threadIdx.x; s < n_seq; s += 64) {
    const int a = seq_offsets ? clamp_off(seq_offsets[s], T) : 0;
    const int b = seq_offsets ? clamp_off(seq_offsets[s + 1], T) : T;
    if (b <= a) continue;
    const double n = b - a;
    double v = 0.0;
    const double* row = term + static_cast<int64_t>(s) * (blocks + 1);
    for (int q = 0; q < blocks; ++q) v += row[q];
    bsum += v * E / (k * n * n);
    zsum += row[blocks];
    filled += 1;
    covered += b - a;
  }
  bsum = wave_sum(bsum);
  zsum = wave_sum(zsum);
  filled = wave_sum(filled);
  covered = wave_sum(covered);
  if (threadIdx.x == 0) {
    losses[0] = filled ? static_cast<float>(bsum / filled) : 0.0f;
    losses[1] = covered ? static_cast<float>(zsum / covered) : 0.0f;
  }
}

// VPL: experts per lane, the least power of two that covers E with 64 lanes.
// Workgroups of a launch over tokens: more rows than this are walked in strides
// (a launch holds fewer than 2^32 threads).
constexpr int64_t kMaxGrid = int64_t(1) << 20;
unsigned token_grid(int64_t n) { return static_cast<unsigned>(n < kMaxGrid ? n : kMaxGrid); }

template <typename F>
hipError_t by_width(int E, F&& f) {
  if (E <= 64) return f(std::integral_constant<int, 1>{});
  if (E <= 128) return f(std::integral_constant<int, 2>{});
  if (E <= 256) return f(std::integral_constant<int, 4>{});
  if (E <= 512) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_select(const SelectOpts& o, const float* logits, const float* balance_bias, int64_t T, int E, int k,
                         int32_t* idx, float* w, hipStream_t s) {
  return by_width(E, [&](auto v) {
    hipLaunchKernelGGL((select_kernel<decltype(v)::value>), dim3(token_grid(T)), dim3(64), 0, s, o, logits,
                       balance_bias, static_cast<int>(T), E, k, idx, w);
    return hipGetLastError();
  });
}

hipError_t launch_select_backward(const SelectOpts& o, const float* logits, const int32_t* idx, const float* w,
                                  const float* dw, const float* dlosses, const int32_t* load,
                                  const int32_t* seq_offsets, int n_seq, int64_t T, int E, int k, float* dlogits,
                                  hipStream_t s) {
  return by_width(E, [&](auto v) {
    hipLaunchKernelGGL((select_backward_kernel<decltype(v)::value>), dim3(token_grid((T + 3) / 4)),
                       dim3(256), 0, s, o, logits, idx, w, dw, dlosses, load, seq_offsets, n_seq, static_cast<int>(T),
                       E, k, dlogits);
    return hipGetLastError();
  });
}

int balance_parts(int64_t T, int n_seq) {
  // about 512 workgroups in all, but no fewer than 16 rows to each
  int64_t parts = (T + 16 * static_cast<int64_t>(n_seq) - 1) / (16 * static_cast<int64_t>(n_seq));
  const int64_t most = 512 / n_seq;
  if (parts > most) parts = most;
  return parts < 1 ? 1 : static_cast<int>(parts);
}
int balance_blocks(int E) { return (E + kRedE - 1) / kRedE; }

hipError_t launch_balance(const SelectOpts& o, const float* logits, const int32_t* idx, const int32_t* seq_offsets,
                          int n_seq, int64_t T, int E, int k, int parts, float* part_p, int32_t* part_f,
                          double* part_z, double* term, float* losses, int32_t* load, hipStream_t s) {
  const int Ti = static_cast<int>(T), blocks = balance_blocks(E);
  const hipError_t st = by_width(E, [&](auto v) {
    hipLaunchKernelGGL((balance_part_kernel<decltype(v)::value>), dim3(parts, n_seq), dim3(256), 0, s, o, logits, idx,
                       seq_offsets, Ti, E, k, part_p, part_f, part_z);
    return hipGetLastError();
  });
  if (st != hipSuccess) return st;
  hipLaunchKernelGGL(balance_reduce_kernel, dim3(blocks, n_seq), dim3(256), 0, s, part_p, part_f, part_z, parts, E,
                     term, load);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  hipLaunchKernelGGL(balance_final_kernel, dim3(1), dim3(64), 0, s, term, seq_offsets, n_seq, Ti, E, k, blocks,
                     losses);
  return hipGetLastError();
}

}  // namespace moe
