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

// Butterflies over the wave without LDS: lane distances 1, 2 (quad permutes), 4
// (half-row mirror: the quads are uniform by then), 8 (row rotation), 16 and 32
// (row swaps). After each step the lanes it joined hold the same value.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  // every lane has a source, so the old value and bound_ctrl do not matter; this
  // form folds into the instruction that takes the result
  return __builtin_amdgcn_update_dpp(0, v, kCtrl, 0xf, 0xf, true);
}
template <int kDist>
__device__ __forceinline__ void partner(uint32_t v, uint32_t& a, uint32_t& b) {
  if constexpr (kDist == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    a = r[0]; b = r[1];
  } else if constexpr (kDist == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0]; b = r[1];
  } else {
    a = v;
    b = dpp<kDist == 1 ? 0xB1 : kDist == 2 ? 0x4E : kDist == 4 ? 0x141 : 0x128>(v);
  }
}
template <int kDist>
__device__ __forceinline__ void partner_of(float v, float& a, float& b) {
  uint32_t x, y;
  partner<kDist>(__float_as_uint(v), x, y);
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}
template <int kDist>
__device__ __forceinline__ void partner_of(double v, double& a, double& b) {
  uint32_t lx, ly, hx, hy;
  partner<kDist>(static_cast<uint32_t>(__double2loint(v)), lx, ly);
  partner<kDist>(static_cast<uint32_t>(__double2hiint(v)), hx, hy);
  a = __hiloint2double(static_cast<int>(hx), static_cast<int>(lx));
  b = __hiloint2double(static_cast<int>(hy), static_cast<int>(ly));
}
template <int kDist, typename Op>
__device__ __forceinline__ float step_f(float v, Op op) {
  uint32_t a, b;
  partner<kDist>(__float_as_uint(v), a, b);
  return op(__uint_as_float(a), __uint_as_float(b));
}
template <typename Op>
__device__ __forceinline__ float wave_all(float v, Op op) {
  v = step_f<1>(v, op);
  v = step_f<2>(v, op);
  v = step_f<4>(v, op);
  v = step_f<8>(v, op);
  v = step_f<16>(v, op);
  return step_f<32>(v, op);
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_all(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_all(v, [](float a, float b) { return a + b; });
}
template <typename F>
__device__ __forceinline__ F wave_sum_any(F v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
template <int kDist>
__device__ __forceinline__ uint32_t max_step(uint32_t v) {
  uint32_t a, b;
  partner<kDist>(v, a, b);
  return a > b ? a : b;
}
template <int kDist>
__device__ __forceinline__ uint32_t min_step(uint32_t v) {
  uint32_t a, b;
  partner<kDist>(v, a, b);
  return a < b ? a : b;
}
// LDS written by this wave is readable by its other lanes.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int off) {
  const uint32_t lo = __shfl_xor(static_cast<uint32_t>(v), off), hi = __shfl_xor(static_cast<uint32_t>(v >> 32), off);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

// e^x within 2 units in the last place for x <= 88 (0 below -200, -inf and NaN
// included): 2^t of the rounded product t = x log2 e, corrected by what the
// product lost.
__device__ __forceinline__ float exp_fast(float x) {
  x = fmaxf(x, -200.0f);
  const float t = x * 1.44269504f;
  float r = __builtin_fmaf(x, 1.44269504f, -t);
  r = __builtin_fmaf(x, 1.92596299e-8f, r);
  const float p = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(p * r, 0.69314718f, p);
}
// 1 / d for finite d >= 1: the hardware's reciprocal and one Newton step
__device__ __forceinline__ float recip(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}
// s = sigmoid(l) and 1 - s, neither by cancellation
struct Sig {
  float s, n;
};
__device__ __forceinline__ Sig sigmoid2(float l) {
  const float t = exp_fast(-fabsf(l)), r = recip(1.0f + t), q = t * r;
  return l >= 0.0f ? Sig{r, q} : Sig{q, r};
}
// sigmoid(l) / exp(min(m, 0)) for l <= m, with u = exp(l - m): no underflow
// where all of a row's scores are tiny, since only ratios of them are used.
__device__ __forceinline__ float sigmoid_scaled(const Sig& g, float u, float m) { return m >= 0.0f ? g.s : u * g.n; }

// A lane's experts: lane + 64 i, i < VPL, so that a wave's loads and stores are
// whole lines wherever the row starts. Those of i < VPL / 2 exist (by_width).
__device__ __forceinline__ int expert_of(int i) { return (threadIdx.x & 63) + 64 * i; }
template <int VPL>
__device__ __forceinline__ bool has_expert(int i, int E) {
  return (VPL > 1 && i < VPL / 2) || expert_of(i) < E;
}
template <int VPL>
__device__ __forceinline__ void load_raw(const float* __restrict__ row, int E, float pad, float (&v)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool has = has_expert<VPL>(i, E);
    const float u = row[VPL > 1 && i < VPL / 2 ? expert_of(i) : min(expert_of(i), E - 1)];
    v[i] = has ? u : pad;
  }
}
template <int VPL>
__device__ __forceinline__ void clean_row(float (&l)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = live_value(l[i]) ? fminf(l[i], kF32Max) : -INFINITY;
}
template <int VPL>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, float (&l)[VPL]) {
  load_raw<VPL>(row, E, -INFINITY, l);
  clean_row<VPL>(l);
}

template <int VPL>
__device__ __forceinline__ void load_bias(const float* __restrict__ bias, int E, float (&b)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) b[i] = 0.0f;
  if (bias) load_raw<VPL>(bias, E, 0.0f, b);
}

// LDS of one wave.
template <int VPL>
struct __attribute__((aligned(16))) SelectLds {
  uint64_t key[64 * VPL];  // keys by expert; or the candidates' logits and experts, then the best of them
  float val[64 * VPL];     // chosen slots' logits (NaN: out of the choice); or the candidates' keys
};

// Weights of chosen logits v (NaN or -inf: out of the choice) in fp32; a
// renormalised weight is a ratio, formed from scores scaled by the largest
// chosen one (mx). m, inv_z: the row's largest logit and 1 / sum exp(l - m).
__device__ __forceinline__ float weigh(const SelectOpts& o, float v, float mx, float m, float inv_z) {
  if (!live_value(v)) return 0.0f;
  if (o.renorm) {
    const float u = exp_fast(v - mx);
    return o.sigmoid ? sigmoid_scaled(sigmoid2(v), u, mx) : u;
  }
  return o.sigmoid ? sigmoid2(v).s : exp_fast(v - m) * inv_z;
}
__device__ __forceinline__ float weight_factor(const SelectOpts& o, float tot) {
  return o.renorm ? (tot > 0.0f ? o.scale / tot : 0.0f) : o.scale;
}

// The selection by the definition, for any k: double keys, groups ranked from
// LDS, then k rounds of a wave arg-max over (key, logit, lower expert).
template <int VPL>
__device__ __forceinline__ void select_exact(const SelectOpts& o, const float* __restrict__ row,
                                             const float* __restrict__ bias, int E, int k,
                                             int32_t* __restrict__ idx, float* __restrict__ w, SelectLds<VPL>& sh) {
  const int lane = threadIdx.x & 63;
  float l[VPL];
  load_row<VPL>(row, E, l);
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
    zs = wave_sum_any(zs);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float b = bias && has_expert<VPL>(i, E) ? bias[expert_of(i)] : 0.0f;
    const bool live = live_value(l[i]) && live_value(b);
    double s = 0.0;
    if (live) s = o.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l[i]))) : z[i] / zs;
    key[i] = !has_expert<VPL>(i, E) ? kKeyTaken : (live ? order_bits(s + b) : kKeyDead);
  }

  if (o.groups > 1) {
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < VPL; ++i) sh.key[expert_of(i)] = key[i];
    wave_lds_sync();
    const int per = o.per;
    // lane g: group g's key, again as ordered bits (0: no live expert)
    uint64_t gk = 0;
    if (lane < o.groups) {
      uint64_t a = 0, b = 0;
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        const uint64_t v = sh.key[e];
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
      const uint64_t v = (static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(gk >> 32), g)) << 32) |
                         static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(gk), g));
      rank += v > gk || (v == gk && g < lane);
    }
    const uint64_t kept = __ballot(lane < o.groups && rank < o.topk_groups);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (has_expert<VPL>(i, E) && !((kept >> (expert_of(i) / per)) & 1)) key[i] = kKeyDead;
  }

  wave_lds_sync();
  for (int j = 0; j < k; ++j) {
    uint64_t bk = kKeyTaken;
    float bl = 0.0f;
    int be = E;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > bk || (key[i] == bk && key[i] > kKeyDead && l[i] > bl)) { bk = key[i]; bl = l[i]; be = expert_of(i); }
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
      if (expert_of(i) == be) key[i] = kKeyTaken;
    if (lane == 0) {
      idx[j] = be;
      sh.val[j] = bk > kKeyDead ? bl : NAN;
    }
  }
  wave_lds_sync();

  float mx = -INFINITY;
  for (int j = lane; j < k; j += 64) mx = fmaxf(mx, live_value(sh.val[j]) ? sh.val[j] : -INFINITY);
  mx = wave_max(mx);
  const float inv_z = o.sigmoid ? 1.0f : static_cast<float>(1.0 / zs);
  float tot = 0.0f;
  if (o.renorm) {
    for (int j = lane; j < k; j += 64) tot += weigh(o, sh.val[j], mx, m, inv_z);
    tot = wave_sum(tot);
  }
  const float f = weight_factor(o, tot);
  for (int j = lane; j < k; j += 64) w[j] = weigh(o, sh.val[j], mx, m, inv_z) * f;
  wave_lds_sync();
}

// fp32 order bits: larger values, larger integers (-0 as +0).
__device__ __forceinline__ uint32_t order32(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order32_back(uint32_t q) {
  return __uint_as_float(q ^ ((q >> 31) ? 0x80000000u : 0xffffffffu));
}

// The eight lane classes of select_fast bound eight keys. Larger k take select_exact,
// k rounds over the whole row: 4096 x 512 5.8 us with k = 8, 24.3 with 9, 26.1 with 10;
// 4096 x 256 29.3 with k = 16, 4096 x 1024 128 with k = 32.
constexpr int kFastK = 8;
// Error of an fp32 key c = s + bias: at most es + 2^-23 |c|. Sigmoid: s comes out
// of an exponential whose argument is rounded (|l| 2^-24 of it, times s (1 - s):
// below 2^-25), of the exponential, an addition and a reciprocal, 2^-23 or less of
// s or of s (1 - s) each: below 2^-21. Softmax: no score is above inv_z = 1 / sum
// exp(l - m), and a score's error is below 2^-18 of that: argument, exponential,
// reciprocal and product together 2^-20, the sum over at most 16 + 6 additions
// and its terms' own errors 33 2^-24. The sum s + bias rounds by 2^-24 |c|.
__device__ __forceinline__ float score_error(const SelectOpts& o, float inv_z) {
  return o.sigmoid ? 0x1p-21f : 0x1p-18f * inv_z;
}
// two keys near c this far apart are in their exact order
__device__ __forceinline__ float margin(float es, float c) { return 2.0f * (es + 0x1p-23f * fabsf(c)); }

// Groups kept, as a mask with bit g * lpg set: 64 / groups lanes (lpg, a power of
// two) scan a group's keys (c: this lane's, -inf out of the choice) and join.
// `sure` turns false when fp32 keys cannot tell the last kept from the next.
template <typename V, int VPL>
__device__ __forceinline__ uint64_t keep_groups(const SelectOpts& o, const V (&c)[VPL], int per, int lpg, float es,
                                                V* sh, bool& sure) {
  const int lane = threadIdx.x & 63;
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < VPL; ++i) sh[expert_of(i)] = c[i];
  wave_lds_sync();
  const auto most = [](V x, V y) { return x > y ? x : y; };
  const auto least = [](V x, V y) { return x > y ? y : x; };
  const int g = lane >> o.lpg_log2, j = lane & (lpg - 1);
  V a = -INFINITY, b = -INFINITY;
  if (g < o.groups)
    for (int e = j; e < per; e += lpg) {
      const V v = sh[g * per + e];
      b = most(b, least(a, v));
      a = most(a, v);
    }
  auto join = [&](auto dist) {
    constexpr int D = decltype(dist)::value;
    if (lpg > D) {
      V a0, a1, b0, b1;
      partner_of<D>(a, a0, a1);
      partner_of<D>(b, b0, b1);
      b = most(least(a0, a1), most(b0, b1));
      a = most(a0, a1);
    }
  };
  join(std::integral_constant<int, 1>{});
  join(std::integral_constant<int, 2>{});
  join(std::integral_constant<int, 4>{});
  join(std::integral_constant<int, 8>{});
  join(std::integral_constant<int, 16>{});
  join(std::integral_constant<int, 32>{});
  const bool both = o.top2 && b > -INFINITY;
  const V gk = both ? a + b : a;
  // A group's rank: its lanes compare it with lpg groups at a time, and the bits
  // of the ballot that are theirs count.
  int rank = 0;
  const uint64_t own = (~uint64_t(0) >> (64 - lpg)) << (lane - j);
  for (int q0 = 0; q0 < o.groups; q0 += lpg) {
    const int q = q0 + j;
    const V v = __shfl(gk, (q << o.lpg_log2) & 63);
    rank += __popcll(__ballot(q < o.groups && (v > gk || (v == gk && q < g))) & own);
  }
  const bool head = j == 0 && g < o.groups;
  if constexpr (sizeof(V) == 4) {
    // A key is sure of its side when its error does not reach the middle between the
    // last kept key and the next. Every group is asked, not those two alone: biases
    // that cancel give an ordinary key an error of their own size, at any rank. (Groups
    // with nothing live come last in any case, and among each other by their number.)
    const float err = both ? 2.0f * es + 0x1p-22f * (fabsf(a) + fabsf(b)) : es + 0x1p-23f * fabsf(a);
    const auto of_rank = [&](int r) {
      const uint64_t mask = __ballot(head && rank == r);
      return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gk), __ffsll(static_cast<unsigned long long>(mask)) - 1));
    };
    const float middle = 0.5f * of_rank(o.topk_groups - 1) + 0.5f * of_rank(o.topk_groups);
    const bool clear = !(a > -INFINITY) || (rank < o.topk_groups ? gk - err > middle : gk + err < middle);
    sure = !__ballot(head && !clear);
  }
  return __ballot(head && rank < o.topk_groups);
}

// A cut that k to 64 of the wave's keys q reach, by bisection from one that more
// reach; false where equal keys leave none.
template <int VPL>
__device__ __forceinline__ bool nearer_cut(const uint32_t (&q)[VPL], int k, uint32_t& cut) {
  uint32_t lo = __builtin_amdgcn_readfirstlane(cut), hi = 0xffffffffu;  // too many, too few
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    int n = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) n += __popcll(__ballot(q[i] >= mid));
    if (n >= k && n <= 64) {
      cut = mid;
      return true;
    }
    (n < k ? hi : lo) = mid;
  }
  return false;
}

// The same selection for k <= 8 from fp32 keys, one wave per token. Returns
// false (nothing written) for rows with too few experts in the choice, or too
// many equal ones, to bound the candidates; the caller then takes select_exact.
//
// Candidates: the lanes fall into 8 classes (lane mod 8), and the smallest of
// the classes' largest keys has at least 8 keys at or above it; only the keys
// down to there (8 H_8 = 22 of them on average) are ranked, one per lane, by
// counting the larger ones. Where they are more than 64 (one row of 256 experts
// in a thousand: a class whose keys are all small) a nearer cut is looked for.
//
// Without bias and groups the key is the logit itself and the order exact. With
// them it is the fp32 score plus the bias: where a chosen expert's key is within
// its error of a lower one's (about one row in a thousand), the candidates' keys
// are formed again in doubles and ranked by those; likewise the groups' keys
// where the last kept and the next are that close.
template <int VPL, bool kKeyed>
__device__ __forceinline__ bool select_fast(const SelectOpts& o, const float (&raw)[VPL], const float (&bv)[VPL],
                                            const float* __restrict__ bias, int E, int k, int32_t* __restrict__ idx, float* __restrict__ w,
                                            SelectLds<VPL>& sh) {
  const int lane = threadIdx.x & 63;
  float l[VPL], c[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = raw[i];
  clean_row<VPL>(l);

  // the row's largest logit and 1 / sum exp(l - m), where scores need them
  float m = 0.0f, inv_z = 0.0f;
  if (!o.sigmoid && (kKeyed || !o.renorm)) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
    float zs = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      c[i] = exp_fast(l[i] - m);
      zs += c[i];
    }
    zs = wave_sum(zs);
    inv_z = zs > 0.0f ? recip(zs) : 0.0f;  // the largest term is 1
  }
  const float es = score_error(o, inv_z);
  // sum exp(l - m) in doubles, and a double key (for a live expert)
  auto exact_sum = [&]() -> double {
    double zs = 0.0;
    if (!o.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (live_value(l[i])) zs += exp(static_cast<double>(l[i]) - m);
      zs = wave_sum_any(zs);
    }
    return zs;
  };
  auto exact_key = [&](float v, float b, double zs) -> double {
    return (o.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(v))) : exp(static_cast<double>(v) - m) / zs) + b;
  };
  // keys; -inf: out of the choice
  if constexpr (kKeyed) {
    if (o.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] *= inv_z;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int live = static_cast<int>(live_value(l[i])) & static_cast<int>(live_value(bv[i]));
      c[i] = live ? c[i] + bv[i] : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = l[i];
  }

  if (kKeyed && o.groups > 1) {
    const int per = o.per, lpg = 1 << o.lpg_log2;
    bool sure = true;
    uint64_t kept = keep_groups<float, VPL>(o, c, per, lpg, es, sh.val, sure);
    if (!sure) {
      const double zs = exact_sum();
      double cd[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        cd[i] = c[i] > -INFINITY ? exact_key(l[i], bias ? bias[expert_of(i)] : 0.0f, zs) : -INFINITY;
      kept = keep_groups<double, VPL>(o, cd, per, lpg, es, reinterpret_cast<double*>(sh.key), sure);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int ge = static_cast<int>((static_cast<float>(expert_of(i)) + 0.5f) * o.inv_per);  // expert / per, below 2^11
      if (!((kept >> ((ge << o.lpg_log2) & 63)) & 1)) c[i] = -INFINITY;
    }
  }

  // candidates
  uint32_t q[VPL], top = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    q[i] = has_expert<VPL>(i, E) ? order32(c[i]) : 0;
    top = q[i] > top ? q[i] : top;
  }
  top = max_step<8>(top);
  top = max_step<16>(top);
  top = max_step<32>(top);
  top = min_step<1>(top);
  top = min_step<2>(top);
  top = min_step<4>(top);
  int n;
  uint2* const cand = reinterpret_cast<uint2*>(sh.key);  // logit and expert
  uint32_t* const cand_key = reinterpret_cast<uint32_t*>(sh.val);
  for (bool again = false;; again = true) {
    float cut = order32_back(top);
    if (kKeyed) cut -= margin(es, cut);
    // (a cut of -inf stays so; NaN, from a class of no experts or +inf, admits all)
    n = 0;
    wave_lds_sync();
    cand_key[lane] = 0;
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool in = has_expert<VPL>(i, E) && !(c[i] < cut);
      const uint64_t mask = __ballot(in);
      const int at = n + lanes_below(mask);
      if (in && at < 64) {
        cand[at] = make_uint2(__float_as_uint(l[i]), expert_of(i));
        cand_key[at] = q[i];
      }
      n += __popcll(mask);
    }
    if (n <= 64) break;
    if (again || !nearer_cut<VPL>(q, k, top)) return false;
  }
  wave_lds_sync();
  const bool mine = lane < n;
  const uint2 own = cand[lane];
  float v = mine ? __uint_as_float(own.x) : -INFINITY;
  const int e = mine ? static_cast<int>(own.y) : 0;
  const uint32_t key = cand_key[lane];
  const float cv = order32_back(key);
  const bool live = mine && cv > -INFINITY;
  int rank = 0;  // larger candidates (the slots behind the last hold 0)
#pragma unroll 2
  for (int r = 0; r < n; r += 4) {
    const u32x4_t kr = *reinterpret_cast<const u32x4_t*>(cand_key + r);
    rank += kr[0] > key;
    rank += kr[1] > key;
    rank += kr[2] > key;
    rank += kr[3] > key;
  }
  // The best k + 1 in order: a chosen lane that is not the one at its rank has an
  // equal beside it; in keyed form the next lower key must be clearly smaller.
  uint2* const best = cand;  // key and lane
  wave_lds_sync();
  if (lane <= k) best[lane] = make_uint2(0, 64);
  wave_lds_sync();
  if (mine && rank <= k) best[rank] = make_uint2(key, lane);
  wave_lds_sync();
  bool unsure = false;
  if (mine && rank < k) {
    unsure = best[rank].y != static_cast<uint32_t>(lane);
    if (kKeyed) unsure |= live && best[rank + 1].x >= order32(cv - margin(es, cv));
  }
  if (__ballot(unsure)) {
    // by exact keys, then by the logits, then by the experts' order
    uint64_t hi = key, lo = static_cast<uint32_t>(E - 1 - e);
    if constexpr (kKeyed) {
      hi = mine ? kKeyDead : kKeyTaken;
      if (bias) {
        const double zs = exact_sum();
        if (live) hi = order_bits(exact_key(v, bias[e], zs));
        if (live) lo |= static_cast<uint64_t>(order32(v)) << 32;
      } else if (live) {
        hi = order32(v);  // scores without a bias have the logits' order
      }
    }
    const auto of_lane = [](uint64_t x, int at) {
      return (static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(x >> 32), at)) << 32) |
             static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(x), at));
    };
    rank = 0;
    for (int r = 0; r < n; ++r) {
      const uint64_t h = of_lane(hi, r), x = of_lane(lo, r);
      rank += h > hi || (h == hi && x > lo);
    }
  }
  const bool chosen = mine && rank < k;
  if (!chosen || !live) v = -INFINITY;
  float mx = 0.0f, tot = 0.0f, f = o.scale;
  if (o.renorm) mx = wave_max(v);
  const float sc = weigh(o, v, mx, m, inv_z);
  if (o.renorm) {
    tot = wave_sum(sc);
    f = weight_factor(o, tot);
  }
  if (chosen) {
    idx[rank] = e;
    w[rank] = sc * f;
  }
  wave_lds_sync();
  return true;
}

// One wave per token (a loop over tokens would put the rare paths' constants and
// divisions in front of every wave: 400 instructions, as many as a row takes).
// Measured: 1 x 256 with groups and bias 3.3 us, 4096 x 256 the same 6.5, 16383 x
// 250 with bias 11.7 (1.4 TB/s of logits). Bound by vector instructions: 475 a row
// with groups, 311 without (11.7 us are 1.4 times their issue at four cycles each).
// A wave takes one row whatever E is: 16384 x 8 5.3 us, 65536 x 8 15.6. Where a bias
// masks whole groups: 4096 x 256 with 5 of 8 groups masked and 4 kept 6.9, 3 kept 5.5.
template <int VPL, bool kKeyed, bool kFast>
__global__ __launch_bounds__(256) void select_kernel(SelectOpts o, const float* __restrict__ logits,
                                                     const float* __restrict__ bias, int T, int E, int k,
                                                     int32_t* __restrict__ idx, float* __restrict__ w) {
  __shared__ SelectLds<VPL> lds[4];
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wv;
  if (t >= T) return;
  const float* row = logits + t * E;
  int32_t* ti = idx + t * k;
  float* tw = w + t * k;
  if constexpr (kFast) {
    float raw[VPL], bv[VPL];
    load_raw<VPL>(row, E, -INFINITY, raw);
    if (kKeyed) load_bias<VPL>(bias, E, bv);
    if (select_fast<VPL, kKeyed>(o, raw, bv, bias, E, k, ti, tw, lds[wv])) return;
  }
  select_exact<VPL>(o, row, bias, E, k, ti, tw, lds[wv]);
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
// Measured: 4096 x 256 7.2 us, 8192 x 16 6.0, 333 x 60 4.2 (a launch by itself takes
// about 2): bound by the latency of loads, reductions and stores behind each other.
// Each row looks its sequence up among all: 65536 x 256 46 us in one sequence, 84 in 1024.
template <int VPL>
__global__ __launch_bounds__(256) void select_backward_kernel(SelectOpts o, const float* __restrict__ logits,
                                                              const int32_t* __restrict__ idx,
                                                              const float* __restrict__ w,
                                                              const float* __restrict__ dw,
                                                              const float* __restrict__ dlosses,
                                                              const int32_t* __restrict__ load,
                                                              const int32_t* __restrict__ seq_offsets, int n_seq,
                                                              int64_t t0, int T, int E, int k,
                                                              float* __restrict__ dlogits) {
  __shared__ float slots[4][64 * VPL];  // the chosen experts' part, by expert
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* slot = slots[wv];
  const bool need_p = dlosses || !(o.sigmoid || o.renorm);  // softmax over the row
  const int64_t t = t0 + static_cast<int64_t>(blockIdx.x) * 4 + wv;
  if (t >= T) return;
  const int64_t row = t * E, a0 = t * k;
  float l[VPL], dl[VPL], u[VPL];
  Sig g[VPL];
  load_raw<VPL>(logits + row, E, -INFINITY, l);
  // the first 64 slots, loaded beside the row
  int se = -1;
  float sw = 0.0f, sd = 0.0f;
  if (dw && lane < k) {
    se = idx[a0 + lane];
    sw = w[a0 + lane];
    sd = dw[a0 + lane];
  }
  clean_row<VPL>(l);
  float m = 0.0f, zs = 0.0f, inv_z = 0.0f;
  if (need_p) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      u[i] = exp_fast(l[i] - m);
      zs += u[i];
    }
    zs = wave_sum(zs);
    inv_z = zs > 0.0f ? recip(zs) : 0.0f;
  }
  if (o.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) g[i] = live_value(l[i]) ? sigmoid2(l[i]) : Sig{0.0f, 0.0f};
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) dl[i] = 0.0f;

  // the selection
  if (dw) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) slot[expert_of(i)] = 0.0f;
    wave_lds_sync();
    float dsum = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 64) {
      if (j0 > 0) {
        const bool in = j0 + lane < k;
        se = in ? idx[a0 + j0 + lane] : -1;
        sw = in ? w[a0 + j0 + lane] : 0.0f;
        sd = in ? dw[a0 + j0 + lane] : 0.0f;
      }
      // a slot of weight 0 passes nothing on, whatever its dw
      float v = sw != 0.0f ? sw * sd : 0.0f;
      dsum += v;
      if (o.renorm) {
        // dw_j - sum_i v_i dw_i as sum_i v_i (dw_j - dw_i), v = w / scale summing to 1: nothing
        // cancels (divided one by one: 1 / scale is past fp32's range for scales below 2^-128)
        float acc = 0.0f;
        for (int i0 = 0; i0 < k; i0 += 64) {
          const bool in = i0 + lane < k;
          float wi = sw, di = sd;
          if (i0 != j0) {
            wi = in ? w[a0 + i0 + lane] : 0.0f;
            di = in ? dw[a0 + i0 + lane] : 0.0f;
          }
          if (wi == 0.0f) di = 0.0f;
          else wi /= o.scale;
          const int n = min(64, k - i0);
          for (int q = 0; q < n; ++q) {
            const float wq = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wi), q));
            const float dq = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(di), q));
            acc += wq * (sd - dq);
          }
        }
        v = sw != 0.0f ? sw * acc : 0.0f;
      }
      if (se >= 0 && se < E) atomicAdd(&slot[se], v);
    }
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < VPL; ++i) dl[i] = slot[expert_of(i)];
    if (o.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) dl[i] *= g[i].n;
    } else if (!o.renorm) {
      dsum = wave_sum(dsum) * inv_z;
#pragma unroll
      for (int i = 0; i < VPL; ++i) dl[i] -= u[i] * dsum;
    }
  }

  // the losses
  if (dlosses) {
    const Seq q = find_seq(seq_offsets, n_seq, static_cast<int>(t), T);
    if (q.id >= 0 && m > -INFINITY) {
      const float n = static_cast<float>(q.len);
      // (dlosses[0] comes in last: its product with E alone could leave fp32's range)
      const float db = dlosses[0];
      const float cb = static_cast<float>(E) / (static_cast<float>(k) * static_cast<float>(q.filled)) / n / n;
      float f[VPL];  // the loads' bits
      load_raw<VPL>(reinterpret_cast<const float*>(load + static_cast<int64_t>(q.id) * E), E, 0.0f, f);
      // shares p~, up to the factor r
      float sh[VPL], r = inv_z;
      if (o.sigmoid) {
        float tot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          sh[i] = sigmoid_scaled(g[i], u[i], m);
          tot += sh[i];
        }
        r = 1.0f / wave_sum(tot);
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) sh[i] = u[i];
      }
      float gl[VPL], dot = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        sh[i] *= r;
        gl[i] = db * (cb * static_cast<float>(__float_as_int(f[i])));
        dot += sh[i] * gl[i];
      }
      dot = wave_sum(dot);
      // kept finite, so that an expert of share 0 gets 0 where lse is the largest logit
      // there is; but not where the gradient that comes in is no finite number itself
      const float dz = dlosses[1];
      float cz = dz * 2.0f / static_cast<float>(q.covered) * (m + logf(zs)) * inv_z;
      if (fabsf(dz) <= kF32Max) cz = fminf(fmaxf(cz, -kF32Max), kF32Max);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float v = sh[i] * (gl[i] - dot);
        if (o.sigmoid) v *= g[i].n;
        dl[i] += v + cz * u[i];
      }
    }
  }
  // (out of the choice: 0 times a gradient that is no finite number would be NaN)
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (has_expert<VPL>(i, E)) dlogits[row + expert_of(i)] = live_value(l[i]) ? dl[i] : 0.0f;
}

// ---------------------------------------------------------------- losses ----
// Part r of sequence s: its rows' shares p~ summed per expert in double (a part
// of a batch of millions of rows has thousands to a wave) and rounded once to
// fp32, the loads counted (integers, any order gives the same), and sum lse^2 in
// double. The parts are then summed in double. Measured: 4096 x 256 8.2 us and 6 to 7
// for the reduction, 8192 x 16 4.8 and 6.5: latency, as above. Every sequence has the
// same number of parts, so the longest of many takes the time: 8126 x 256 in 64 even
// sequences 35 us (both kernels), with one of 8000 rows 129; 65536 x 256 as one
// sequence 39, in 1024 of 64 rows 388, with one of 60000 rows among 1024 short ones
// 13200.
template <int VPL>
__global__ __launch_bounds__(256) void balance_part_kernel(SelectOpts o, const float* __restrict__ logits,
                                                           const int32_t* __restrict__ idx,
                                                           const int32_t* __restrict__ seq_offsets, int T, int E, int k,
                                                           float* __restrict__ part_p, int32_t* __restrict__ part_f,
                                                           double* __restrict__ part_z, uint32_t* __restrict__ done) {
  __shared__ int32_t cnt[64 * VPL];
  __shared__ double psum[4][64 * VPL];
  __shared__ double zsum[4];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = blockIdx.x, s = blockIdx.y, parts = gridDim.x;
  if (r == 0 && s == 0 && threadIdx.x == 0) *done = 0;
  const int a = seq_offsets ? clamp_off(seq_offsets[s], T) : 0, b = seq_offsets ? clamp_off(seq_offsets[s + 1], T) : T;
  const int64_t n = b > a ? b - a : 0;
  const int lo = a + static_cast<int>(n * r / parts), hi = a + static_cast<int>(n * (r + 1) / parts);
  for (int e = threadIdx.x; e < 64 * VPL; e += 256) cnt[e] = 0;
  __syncthreads();
  double acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0;
  double zacc = 0.0;
  // two rows at a time: their loads and their reductions' latencies overlap
  for (int64_t t = lo + wv; t < hi; t += 8) {
    float l[2][VPL], x[2][VPL], m[2], zs[2], tot[2];
    int32_t e[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool on = t + 4 * u < hi;
      const int64_t row = on ? t + 4 * u : t;
      load_raw<VPL>(logits + row * E, E, -INFINITY, l[u]);
      e[u] = on && lane < k ? idx[row * k + lane] : -1;
      for (int j = lane + 64; on && j < k; j += 64) {
        const int q = idx[row * k + j];
        if (q >= 0 && q < E) atomicAdd(&cnt[q], 1);
      }
      if (!on) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[u][i] = -INFINITY;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (e[u] >= 0 && e[u] < E) atomicAdd(&cnt[e[u]], 1);
      clean_row<VPL>(l[u]);
      m[u] = l[u][0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) m[u] = fmaxf(m[u], l[u][i]);
      m[u] = wave_max(m[u]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      zs[u] = tot[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        x[u][i] = exp_fast(l[u][i] - m[u]);
        zs[u] += x[u][i];
        if (o.sigmoid) {
          x[u][i] = live_value(l[u][i]) ? sigmoid_scaled(sigmoid2(l[u][i]), x[u][i], m[u]) : 0.0f;
          tot[u] += x[u][i];
        }
      }
      zs[u] = wave_sum(zs[u]);
      tot[u] = o.sigmoid ? wave_sum(tot[u]) : zs[u];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (m[u] == -INFINITY) continue;  // nothing in the choice, or no row
      const float r = 1.0f / tot[u];
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] += x[u][i] * r;
      const double lse = static_cast<double>(m[u]) + logf(zs[u]);
      zacc += lse * lse;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) psum[wv][expert_of(i)] = acc[i];
  if (lane == 0) zsum[wv] = zacc;
  __syncthreads();
  const int64_t base = (static_cast<int64_t>(s) * parts + r) * E;
  for (int e = threadIdx.x; e < E; e += 256) {
    part_p[base + e] = static_cast<float>(((psum[0][e] + psum[1][e]) + psum[2][e]) + psum[3][e]);
    part_f[base + e] = cnt[e];
  }
  if (threadIdx.x == 0) part_z[static_cast<int64_t>(s) * parts + r] = ((zsum[0] + zsum[1]) + zsum[2]) + zsum[3];
}

constexpr int kRedE = 16;  // experts per block of the part reduction

// Block (eb, s): parts summed in order for kRedE experts (16 slices of parts,
// then the slices in order), load[s][e] written, the experts' terms f * P added
// into term[s][eb]; term[s][blocks] holds the sequence's sum of lse^2. The block
// that finishes last (a counter the part kernel cleared) adds the terms in order:
// B = 1/filled sum_s E / (k n_s^2) sum_e f P, Z = sum lse^2 / covered.
__global__ __launch_bounds__(256) void balance_reduce_kernel(const float* __restrict__ part_p,
                                                             const int32_t* __restrict__ part_f,
                                                             const double* __restrict__ part_z, int parts,
                                                             const int32_t* __restrict__ seq_offsets, int n_seq, int T,
                                                             int E, int k, double* term, int32_t* __restrict__ load,
                                                             uint32_t* done, float* __restrict__ losses) {
  __shared__ double sp[16][kRedE];
  __shared__ int32_t sf[16][kRedE];
  __shared__ double sz[4];
  __shared__ bool last;
  const int blocks = gridDim.x;
  const int s = blockIdx.y, el = threadIdx.x % kRedE, sl = threadIdx.x / kRedE;
  const int e = blockIdx.x * kRedE + el;
  double p = 0.0;
  int32_t f = 0;
  if (e < E) {
    const int64_t base = static_cast<int64_t>(s) * parts * E + e;
#pragma unroll 8
    for (int r = sl; r < parts; r += 16) {
      p += part_p[base + static_cast<int64_t>(r) * E];
      f += part_f[base + static_cast<int64_t>(r) * E];
    }
  }
  sp[sl][el] = p;
  sf[sl][el] = f;
  double z = 0.0;
  if (blockIdx.x == 0) {
    for (int r = threadIdx.x; r < parts; r += 256) z += part_z[static_cast<int64_t>(s) * parts + r];
    z = wave_sum_any(z);
    if ((threadIdx.x & 63) == 0) sz[threadIdx.x >> 6] = z;
  }
  __syncthreads();
  if (threadIdx.x < kRedE) {
    double ps = 0.0;
    int32_t fs = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) { ps += sp[q][threadIdx.x]; fs += sf[q][threadIdx.x]; }
    if (e < E) load[static_cast<int64_t>(s) * E + e] = fs;
    double v = ps * fs;
#pragma unroll
    for (int off = kRedE / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, kRedE);
    if (threadIdx.x == 0) {
      double* row = term + static_cast<int64_t>(s) * (blocks + 1);
      row[blockIdx.x] = v;
      if (blockIdx.x == 0) row[blocks] = ((sz[0] + sz[1]) + sz[2]) + sz[3];
      __threadfence();
      last = atomicAdd(done, 1u) == gridDim.x * gridDim.y - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double bsum = 0.0, zsum = 0.0;
  int filled = 0, covered = 0;
  const int64_t terms = static_cast<int64_t>(n_seq) * (blocks + 1);
  for (int64_t x = threadIdx.x; x < terms; x += 256) {
    const int q = static_cast<int>(x / (blocks + 1)), at = static_cast<int>(x % (blocks + 1));
    const int a = seq_offsets ? clamp_off(seq_offsets[q], T) : 0;
    const int b = seq_offsets ? clamp_off(seq_offsets[q + 1], T) : T;
    if (b <= a) continue;
    const double v = __hip_atomic_load(term + x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const double n = b - a;
    if (at < blocks) {
      bsum += v * E / (k * n * n);
    } else {
      zsum += v;
      filled += 1;
      covered += b - a;
    }
  }
  __shared__ double sb[4], sv[4];
  __shared__ int si[4], sc[4];
  bsum = wave_sum_any(bsum);
  zsum = wave_sum_any(zsum);
  filled = wave_sum_any(filled);
  covered = wave_sum_any(covered);
  if ((threadIdx.x & 63) == 0) {
    const int q = threadIdx.x >> 6;
    sb[q] = bsum; sv[q] = zsum; si[q] = filled; sc[q] = covered;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    filled = ((si[0] + si[1]) + si[2]) + si[3];
    covered = ((sc[0] + sc[1]) + sc[2]) + sc[3];
    losses[0] = filled ? static_cast<float>((((sb[0] + sb[1]) + sb[2]) + sb[3]) / filled) : 0.0f;
    losses[1] = covered ? static_cast<float>((((sv[0] + sv[1]) + sv[2]) + sv[3]) / covered) : 0.0f;
  }
}

// Tokens of one launch (it holds fewer than 2^32 threads, 64 to a token); a
// larger batch takes several.
constexpr int64_t kLaunchTokens = int64_t(1) << 25;
template <typename F>
hipError_t by_tokens(int64_t T, F&& f) {
  for (int64_t t0 = 0; t0 < T; t0 += kLaunchTokens) {
    const int64_t n = T - t0 < kLaunchTokens ? T - t0 : kLaunchTokens;
    if (const hipError_t st = f(t0, static_cast<int>(n)); st != hipSuccess) return st;
  }
  return hipSuccess;
}

// VPL: experts per lane, the least power of two that covers E with 64 lanes.
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
  return by_tokens(T, [&](int64_t t0, int n) {
    const dim3 grid((n + 3) / 4);
    const float* l = logits + t0 * E;
    int32_t* ti = idx + t0 * k;
    float* tw = w + t0 * k;
    return by_width(E, [&](auto v) {
      constexpr int VPL = decltype(v)::value;
      if (k > kFastK)
        hipLaunchKernelGGL((select_kernel<VPL, true, false>), grid, dim3(256), 0, s, o, l, balance_bias, n, E, k, ti, tw);
      else if (balance_bias || o.groups > 1)
        hipLaunchKernelGGL((select_kernel<VPL, true, true>), grid, dim3(256), 0, s, o, l, balance_bias, n, E, k, ti, tw);
      else
        hipLaunchKernelGGL((select_kernel<VPL, false, true>), grid, dim3(256), 0, s, o, l, balance_bias, n, E, k, ti, tw);
      return hipGetLastError();
    });
  });
}

hipError_t launch_select_backward(const SelectOpts& o, const float* logits, const int32_t* idx, const float* w,
                                  const float* dw, const float* dlosses, const int32_t* load,
                                  const int32_t* seq_offsets, int n_seq, int64_t T, int E, int k, float* dlogits,
                                  hipStream_t s) {
  return by_tokens(T, [&](int64_t t0, int n) {
    return by_width(E, [&](auto v) {
      hipLaunchKernelGGL((select_backward_kernel<decltype(v)::value>), dim3((n + 3) / 4), dim3(256), 0, s, o, logits,
                         idx, w, dw, dlosses, load, seq_offsets, n_seq, t0, static_cast<int>(T), E, k, dlogits);
      return hipGetLastError();
    });
  });
}

int balance_parts(int64_t T, int n_seq, int E) {
  // No fewer than 8 rows (two to a wave) to a part; in all, about 1024 parts, or
  // 512 up to 64 experts, where few workgroups add the parts up: 4096 x 256 took
  // 12.3 + 7.1 us (parts, reduction) with 256 parts and 8.7 + 6.4 with 512;
  // 8192 x 16 took 5.1 + 6.9 us with 512 and 4.8 + 8.9 with 1024.
  int64_t parts = (T + 8 * static_cast<int64_t>(n_seq) - 1) / (8 * static_cast<int64_t>(n_seq));
  const int64_t most = (E > 64 ? 1024 : 512) / n_seq;
  if (parts > most) parts = most;
  return parts < 1 ? 1 : static_cast<int>(parts);
}
int balance_blocks(int E) { return (E + kRedE - 1) / kRedE; }

hipError_t launch_balance(const SelectOpts& o, const float* logits, const int32_t* idx, const int32_t* seq_offsets,
                          int n_seq, int64_t T, int E, int k, int parts, float* part_p, int32_t* part_f,
                          double* part_z, double* term, uint32_t* done, float* losses, int32_t* load,
                          hipStream_t s) {
  const int Ti = static_cast<int>(T), blocks = balance_blocks(E);
  const hipError_t st = by_width(E, [&](auto v) {
    hipLaunchKernelGGL((balance_part_kernel<decltype(v)::value>), dim3(parts, n_seq), dim3(256), 0, s, o, logits, idx,
                       seq_offsets, Ti, E, k, part_p, part_f, part_z, done);
    return hipGetLastError();
  });
  if (st != hipSuccess) return st;
  hipLaunchKernelGGL(balance_reduce_kernel, dim3(blocks, n_seq), dim3(256), 0, s, part_p, part_f, part_z, parts,
                     seq_offsets, n_seq, Ti, E, k, term, load, done, losses);
  return hipGetLastError();
}

}  // namespace moe
