// The gradients' 2-norm over a list of tensors, and the AdamW update of one with
// states in 32 or 8 bits. The contract is in include/moe.h.
#include "common.h"
#include "philox.h"
#include "train.h"

namespace moe {

namespace {

// The tensor of chunk `c` of a launch: lanes compare c with the tensors' first
// chunks (not decreasing), and the last one at or below it is the one.
template <int kMost, typename Table>
__device__ __forceinline__ int find_tensor(const Table& t, uint32_t c) {
  int at = 0;
#pragma unroll
  for (int base = 0; base < kMost; base += 64) {
    const int i = base + static_cast<int>(threadIdx.x & 63);
    const bool below = i < kMost && i < t.count && t.t[i < kMost ? i : 0].first <= c;
    at += __popcll(__ballot(below));
  }
  return __builtin_amdgcn_readfirstlane(at - 1);
}

// kStream: lists of over half the 256 MB cache pass through once, and no cache line
// is kept for them. Measured, ordinary and streaming loads and stores (three lists
// in turn): update of fp32 weights with fp32 states, 4 M (117 MB) 20.5 and 22.0 us,
// 8 M (235 MB) 48 and 42, 64 M 360 and 336; of bf16 weights with 8-bit states, 12 M
// (126 MB) 29 and 31, 16 M 42 and 42, 64 M 145 and 139; 2-norm of fp32 gradients,
// 16 M (67 MB) 16.1 and 16.1, 32 M (134 MB) 28.8 and 26.0, 302 M 198 and 179.
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
template <bool kStream>
__device__ __forceinline__ uint4 load16(const void* p) {
  const u32x4_t* q = static_cast<const u32x4_t*>(p);
  const u32x4_t v = kStream ? __builtin_nontemporal_load(q) : *q;
  return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool kStream>
__device__ __forceinline__ uint2 load2(const void* p) {
  const u32x2_t* q = static_cast<const u32x2_t*>(p);
  const u32x2_t v = kStream ? __builtin_nontemporal_load(q) : *q;
  return make_uint2(v[0], v[1]);
}
template <bool kStream>
__device__ __forceinline__ void put(void* p, const uint4& v) {
  u32x4_t* q = static_cast<u32x4_t*>(p);
  if (kStream) __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, q);
  else *q = u32x4_t{v.x, v.y, v.z, v.w};
}
template <bool kStream>
__device__ __forceinline__ void put(void* p, const uint2& v) {
  u32x2_t* q = static_cast<u32x2_t*>(p);
  if (kStream) __builtin_nontemporal_store(u32x2_t{v.x, v.y}, q);
  else *q = u32x2_t{v.x, v.y};
}

// A thread's place in a turn of the workgroup: eight elements of which `left` exist,
// in two groups of four, from i and from i + kGap. Eight in a row (kGap 4) where
// they share a generator's call or are bf16; else 1024 apart, so that a wave's fp32
// loads and stores are whole lines. wide: the group is there as a whole and its
// buffers are aligned.
template <int kGap_>
struct Place {
  static constexpr int kGap = kGap_;
  int i, left;
  bool wide[2];
  __device__ __forceinline__ Place(int q, int left_, bool aligned) : i(q + threadIdx.x * (kGap == 4 ? 8 : 4)), left(left_) {
    wide[0] = aligned && i + (kGap == 4 ? 8 : 4) <= left;
    wide[1] = kGap == 4 ? wide[0] : aligned && i + kGap + 4 <= left;
  }
};

template <bool kStream, int kGap>
__device__ __forceinline__ void load8(const void* p, bool bf16, const Place<kGap>& c, float (&v)[8]) {
  if (kGap == 4 && bf16 && c.wide[0]) {
    const uint4 u = load16<kStream>(static_cast<const bf16_t*>(p) + c.i);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = c.i + h * kGap;
    float* o = v + 4 * h;
    if (c.wide[h]) {
      if (bf16) {
        const uint2 u = load2<kStream>(static_cast<const bf16_t*>(p) + at);
        o[0] = bf16_lo(u.x); o[1] = bf16_hi(u.x); o[2] = bf16_lo(u.y); o[3] = bf16_hi(u.y);
      } else {
        const uint4 u = load16<kStream>(static_cast<const float*>(p) + at);
        o[0] = __uint_as_float(u.x); o[1] = __uint_as_float(u.y);
        o[2] = __uint_as_float(u.z); o[3] = __uint_as_float(u.w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j] = 0.0f;
        if (at + j < c.left)
          o[j] = bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const bf16_t*>(p)[at + j]) << 16)
                      : static_cast<const float*>(p)[at + j];
      }
    }
  }
}

template <bool kStream, int kGap>
__device__ __forceinline__ void store8(float* p, const Place<kGap>& c, const float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = c.i + h * kGap;
    const float* o = v + 4 * h;
    if (c.wide[h]) {
      put<kStream>(p + at, make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                                      __float_as_uint(o[3])));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at + j < c.left) p[at + j] = o[j];
    }
  }
}

// w: bf16 patterns, element j in the low (even j) or high half of word j / 2
template <bool kStream, int kGap>
__device__ __forceinline__ void store8_bf16(bf16_t* p, const Place<kGap>& c, const uint32_t (&w)[4]) {
  if (kGap == 4 && c.wide[0]) {
    put<kStream>(p + c.i, make_uint4(w[0], w[1], w[2], w[3]));
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = c.i + h * kGap;
    if (c.wide[h]) {
      put<kStream>(p + at, make_uint2(w[2 * h], w[2 * h + 1]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at + j < c.left) p[at + j] = static_cast<bf16_t>(w[2 * h + (j >> 1)] >> (16 * (j & 1)));
    }
  }
}

// First element of a turn in a buffer of either type, and how many it has there.
__device__ __forceinline__ const void* from(const void* p, bool bf16, int64_t i0) {
  return static_cast<const char*>(p) + (bf16 ? 2 : 4) * i0;
}
__device__ __forceinline__ int left_of(int64_t n, int64_t i0, int chunk) {
  return static_cast<int>(n - i0 < chunk ? n - i0 : chunk);
}

__device__ __forceinline__ void round_bf16(const float (&v)[8], uint32_t (&w)[4]) {
  bf16x8_t o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = static_cast<__bf16>(v[j]);
  const uint4 u = *reinterpret_cast<uint4*>(&o);
  w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
}

// ---------------- 2-norm ----------------
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  const int nw = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < nw; ++i) v += red[i];
  __syncthreads();
  return v;
}

template <bool kStream>
__device__ __forceinline__ double chunk_squares(const GradTable& t, uint32_t c) {
  const GradEntry& g = t.t[find_tensor<kGradTensors>(t, c)];
  const bool bf16 = g.flags & 1, aligned = g.flags & 2;
  const int64_t i0 = static_cast<int64_t>(c - g.first) * t.chunk;
  const void* p = from(g.g, bf16, i0);
  const int left = left_of(g.n, i0, t.chunk);
  double s = 0.0;
  for (int q = 0; q < left; q += kRound) {
    float v[8];
    if (bf16) load8<kStream>(p, true, Place<4>(q, left, aligned), v);
    else load8<kStream>(p, false, Place<1024>(q, left, aligned), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), s);
  }
  return s;
}

template <bool kStream>
__global__ __launch_bounds__(256) void square_sums_kernel(GradTable t, double* __restrict__ parts) {
  __shared__ double red[4];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) s += chunk_squares<kStream>(t, c);
  s = block_sum(s, red);
  if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

// A norm that is not finite gives a factor of NaN, which the update takes for "no step".
__device__ __forceinline__ void write_norm(double sum, double scale, double max_norm, float* out) {
  const double norm = sqrt(sum) * fabs(scale);
  const double f = max_norm / (norm + 1e-6);
  out[0] = static_cast<float>(norm);
  out[1] = norm < HUGE_VAL ? static_cast<float>(scale * (f < 1.0 ? f : 1.0)) : __uint_as_float(0x7fc00000u);
}

__global__ __launch_bounds__(1024) void grad_norm_kernel(const double* __restrict__ parts, int n, double scale,
                                                         double max_norm, float* out) {
  __shared__ double red[16];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) s += parts[i];
  s = block_sum(s, red);
  if (threadIdx.x == 0) write_norm(s, scale, max_norm, out);
}

// ---------------- AdamW ----------------
// m and the root of v are held as a byte per element and a scale byte per 128
// elements: the scale is a biased fp32 exponent E (255: not finite, reads as
// NaN), the byte the top bits of the value brought down by 2^(15 - E) to fp32
// exponents 0 .. 15, so that gradual underflow, rounding and decoding are those
// of fp32's own bits. m has a sign and three fraction bits, the root (never
// below 0) four.
__device__ __forceinline__ int row16_max(int v) {
  // over the 16 lanes of a row
  v = max(v, __builtin_amdgcn_mov_dpp(v, 0x128, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_mov_dpp(v, 0x124, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_mov_dpp(v, 0x122, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_mov_dpp(v, 0x121, 0xf, 0xf, false));
  return v;
}

// Codes move between byte 3 of a word and fp32 bits by shifts: a code's magnitude
// is bits 26 .. 20 (m) or 26 .. 19 (root) of the fp32 value.
__device__ __forceinline__ float decode_m(uint32_t word, int j) {
  const int c = static_cast<int>(word << (24 - 8 * (j & 3))) >> 4;
  return __uint_as_float(static_cast<uint32_t>(c) & 0x87f00000u);
}
__device__ __forceinline__ float decode_r(uint32_t word, int j) {
  return __uint_as_float(((word >> (8 * (j & 3))) & 0xffu) << 19);
}

// The scale byte of 128 elements (16 lanes of eight) from each lane's largest
// magnitude, as bits: the exponent whose top code holds the largest of them, 255
// where one is not finite.
template <int kShift>
__device__ __forceinline__ int scale_of(uint32_t top) {
  const uint32_t e = (static_cast<uint32_t>(row16_max(static_cast<int>(top))) + ((1u << kShift) - 1u)) >> 23;
  return static_cast<int>(min(e, 255u));
}

// Byte 3 of four words.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0703u), hi = __builtin_amdgcn_perm(d, c, 0x07030c0cu);
  return lo | hi;
}

// Codes of eight values: rounded by the 16-bit numbers u (up where the dropped
// bits and u reach a step).
__device__ __forceinline__ uint2 encode_m(const float (&x)[8], const uint32_t (&u)[8], int e) {
  uint32_t t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(__builtin_amdgcn_ldexpf(x[j], 15 - e)) + (u[j] << 4);
    t[j] = (b & 0x80000000u) | (b << 4);  // (bit 27 is 0 where the code counts)
  }
  const bool bad = e == 255;
  return make_uint2(bad ? 0u : top_bytes(t[0], t[1], t[2], t[3]), bad ? 0u : top_bytes(t[4], t[5], t[6], t[7]));
}
__device__ __forceinline__ uint2 encode_r(const float (&x)[8], const uint32_t (&u)[8], int e) {
  uint32_t t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(__builtin_amdgcn_ldexpf(x[j], 15 - e)) + (u[j] << 3);
    // a root above 0 stays above 0, as the update divides by it: the median of b, the least code and the root's own
    // bits (which lie above any code's, as roots of fp32 values lie above 2^-75; 0 leaves b, less than a code of u)
    t[j] = __float_as_uint(__builtin_amdgcn_fmed3f(__uint_as_float(b), __uint_as_float(1u << 19), x[j])) << 5;
  }
  const bool bad = e == 255;
  return make_uint2(bad ? 0u : top_bytes(t[0], t[1], t[2], t[3]), bad ? 0u : top_bytes(t[4], t[5], t[6], t[7]));
}

template <bool kStream>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, const Place<4>& c) {
  if (c.wide[0]) return load2<kStream>(p + c.i);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c.i + j < c.left) w[j >> 2] |= static_cast<uint32_t>(p[c.i + j]) << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

template <bool kStream>
__device__ __forceinline__ void store_codes(uint8_t* p, const Place<4>& c, const uint2& v) {
  if (c.wide[0]) {
    put<kStream>(p + c.i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.i + j < c.left) p[c.i + j] = static_cast<uint8_t>((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
  }
}

// Square roots rounded to nearest, 0 for 0, and the largest of them as bits. From
// 2^-96 on (and for 0): the reciprocal root's approximation, its product with v
// corrected by what its square leaves of v. Compared with the rounded roots of
// every fp32 fraction in two binades (all there are, up to powers of 4) it gives
// each of them. Returns whether a lane of the wave has a smaller value, an infinity
// or NaN (the roots are formed the longer way then).
__device__ __forceinline__ bool roots(const float (&v)[8], float (&r)[8], uint32_t& top) {
  constexpr uint32_t kLeast = 31u << 23, kInf = 255u << 23;  // 2^-96, infinity: v is never below 0, NaN lies above
  uint32_t least = 0xffffffffu;
  top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    least = min(least, __float_as_uint(v[j]) - 1u);  // (0 passes)
    const float y = __builtin_amdgcn_rsqf(__uint_as_float(max(__float_as_uint(v[j]), kLeast)));
    const float s = v[j] * y;
    r[j] = fmaf(fmaf(-s, s, v[j]), 0.5f * y, s);
    top = max(top, __float_as_uint(r[j]) & 0x7fffffffu);
  }
  // (an infinity's product with its reciprocal root is NaN)
  if (__ballot(least < kLeast - 1u || top >= kInf) == 0) return false;
  top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    r[j] = sqrtf(v[j]);
    top = max(top, __float_as_uint(r[j]) & 0x7fffffffu);
  }
  return true;
}

// One turn of a workgroup to at most t.chunk elements of a tensor.
// With 32-bit states bound by memory, where fewer, shorter turns at a time keep the
// accesses closer together: 302 M bf16 weights with fp32 masters, states and
// gradients in turns of 2048, at most 3, 4, 5, 6, 8 waves to a SIMD 1541, 1525,
// 1584, 1601, 1616 us; in turns of 4096 1572 and 1601 with 3 and 4, of 8192 1589,
// 1657, 1665, 1678, 1686 with 3, 4, 5, 6, 8 (9.66 GB: 6.3 TB/s at best).
// With 8-bit states by the vector instructions, some 490 to a wave's 512 elements,
// and memory alike: 88 M bf16 weights and gradients 170 us (883 MB, 5.2 TB/s); with
// 4, 5, 6 and 8 waves (and the states read out) 273, 250, 237, 234 us.
template <int kBits, bool kStream>
__global__ __attribute__((amdgpu_waves_per_eu(1, kBits == 32 ? 4 : 8))) __launch_bounds__(256) void adam_kernel(
    AdamTable t) {
#pragma clang fp contract(off)
  const uint32_t c = blockIdx.x;
  const AdamEntry& en = t.t[find_tensor<kAdamTensors>(t, c)];
  AdamScalars k = t.k;
  if (t.lr_step) adam_scalars(k, t.lr_step[0], t.lr_step[1]);
  const float gs = t.gscale ? t.gscale[0] : 1.0f;
  // gradients that are not finite as a whole: no step
  if (!(fabsf(gs) < INFINITY)) return;
  const bool pb = en.flags & kAdamParamBf16, gb = en.flags & kAdamGradBf16, al = en.flags & kAdamAligned;
  const int64_t i0 = static_cast<int64_t>(c - en.first) * t.chunk;
  const int left = left_of(en.n, i0, t.chunk);
  void* const p = const_cast<void*>(from(en.p, pb, i0));
  float* const master = en.master ? en.master + i0 : nullptr;
  const void* const grad = from(en.g, gb, i0);
  const bool sr = t.stochastic && pb && !master;
  uint64_t seed = 0, offset = 0;
  if (t.rng) seed = t.rng[0], offset = t.rng[1];
  const uint64_t first8 = static_cast<uint64_t>(en.base + i0) >> 3;  // (both are multiples of 8)
  constexpr int kGap = kBits == 8 ? 4 : 1024;
  constexpr int kState = kBits == 8 ? 1 : 4;  // bytes of a state's element
  char* const sm = static_cast<char*>(en.m) + kState * i0;
  char* const sv = static_cast<char*>(en.v) + kState * i0;
  uint8_t* const qm = kBits == 8 ? en.ms + i0 / kScaleBlock : nullptr;
  uint8_t* const qv = kBits == 8 ? en.vs + i0 / kScaleBlock : nullptr;
  const float nan = __uint_as_float(0x7fc00000u);
  for (int q = 0; q < left; q += kRound) {
    const Place<kGap> at(q, left, al);
    float w[8], g[8], m[8], v[8];
    if (master) load8<kStream>(master, false, at, w);
    else load8<kStream>(p, pb, at, w);
    load8<kStream>(grad, gb, at, g);
    float b1 = k.b1, b2 = k.b2;
    if constexpr (kBits == 32) {
      load8<kStream>(sm, false, at, m);
      load8<kStream>(sv, false, at, v);
    } else {
      // codes keep the ordinary way: 88 M of them stepped 177 us instead of 175, but stepped and then read out (16
      // bytes an element in all) 240 instead of 267
      const uint2 cm = load_codes<false>(reinterpret_cast<const uint8_t*>(sm), at);
      const uint2 cv = load_codes<false>(reinterpret_cast<const uint8_t*>(sv), at);
      const bool in = at.i < left;
      const int em = in ? qm[at.i / kScaleBlock] : 0, ev = in ? qv[at.i / kScaleBlock] : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = decode_m(j < 4 ? cm.x : cm.y, j);
        const float r = __builtin_amdgcn_ldexpf(decode_r(j < 4 ? cv.x : cv.y, j), ev - 15);
        v[j] = r * r;
      }
      // m's scale goes into beta1 (the product's value and rounding are the same), where it fits there
      if (__ballot(em > 142) == 0) {
        b1 = __builtin_amdgcn_ldexpf(b1, em - 15);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = __builtin_amdgcn_ldexpf(m[j], em - 15);
        if (em == 255) b1 = nan;
      }
      if (ev == 255) b2 = nan;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = g[j] * gs;
      m[j] = m[j] * b1 + x * k.c1;
      v[j] = v[j] * b2 + (x * x) * k.c2;
    }
    float r[8];
    uint32_t top;
    const bool odd = roots(v, r, top);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // (the reciprocal is off by 2^-23 at most, and eps keeps it in range)
      const float up = k.step_size * m[j] * __builtin_amdgcn_rcpf(fmaf(r[j], k.inv_root, k.eps));
      w[j] = w[j] - fmaf(k.decay, w[j], up);
    }
    uint32_t u[8];
    if (kBits == 8 || sr) {
      Philox x = philox(first8 + (at.i >> 3), offset, seed);
      if constexpr (kGap != 4) {
        // each group of four is one half of a call's eight
        const Philox z = philox(first8 + ((at.i + kGap) >> 3), offset, seed);
        const bool upper = at.i & 4;
        x = {{upper ? x.x[2] : x.x[0], upper ? x.x[3] : x.x[1], upper ? z.x[2] : z.x[0], upper ? z.x[3] : z.x[1]}};
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[2 * j] = x.x[j] & 0xffffu;
        u[2 * j + 1] = x.x[j] >> 16;
      }
    }
    if (master) store8<kStream>(master, at, w);
    if (pb) {
      uint32_t o[4];
      if (sr) {
        // Cut after adding the number. Infinities stay: their low bits are 0. So does a NaN of a bf16 weight or of the
        // 8-bit states; others, whose bits might carry over, come with a gradient or a 32-bit state.
        if (kBits == 32 || odd) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = w[j] != w[j] ? nan : w[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = __builtin_amdgcn_perm(__float_as_uint(w[2 * j + 1]) + u[2 * j + 1], __float_as_uint(w[2 * j]) + u[2 * j],
                                       0x07060302u);
      } else {
        round_bf16(w, o);
      }
      store8_bf16<kStream>(static_cast<bf16_t*>(p), at, o);
    } else {
      store8<kStream>(static_cast<float*>(p), at, w);
    }
    if constexpr (kBits == 32) {
      store8<kStream>(reinterpret_cast<float*>(sm), at, m);
      store8<kStream>(reinterpret_cast<float*>(sv), at, v);
    } else {
      // elements past the tensor's end are 0 in every row of 16 lanes
      uint32_t top_m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top_m = max(top_m, __float_as_uint(m[j]) & 0x7fffffffu);
      const int em = scale_of<20>(top_m), ev = scale_of<19>(top);
      store_codes<false>(reinterpret_cast<uint8_t*>(sm), at, encode_m(m, u, em));
      store_codes<false>(reinterpret_cast<uint8_t*>(sv), at, encode_r(r, u, ev));
      if ((threadIdx.x & 15) == 0 && at.i < left) {
        qm[at.i / kScaleBlock] = static_cast<uint8_t>(em);
        qv[at.i / kScaleBlock] = static_cast<uint8_t>(ev);
      }
    }
  }
}

template <int kOut, bool kStream>
__global__ __launch_bounds__(256) void state_values_kernel(StateTable t) {
  const uint32_t c = blockIdx.x;
  const StateEntry& en = t.t[find_tensor<kStateTensors>(t, c)];
  const int64_t i0 = static_cast<int64_t>(c - en.first) * t.chunk;
  const int left = left_of(en.n, i0, t.chunk);
  void* const pm = const_cast<void*>(from(en.m_out, kOut == 1, i0));
  void* const pr = const_cast<void*>(from(en.r_out, kOut == 1, i0));
  const float nan = __uint_as_float(0x7fc00000u);
  for (int q = 0; q < left; q += kRound) {
    const Place<4> at(q, left, en.aligned);
    if (at.i >= left) break;
    const uint2 cm = load_codes<kStream>(en.m + i0, at), cv = load_codes<kStream>(en.v + i0, at);
    const int em = en.ms[(i0 + at.i) / kScaleBlock], ev = en.vs[(i0 + at.i) / kScaleBlock];
    float m[8], r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = em == 255 ? nan : __builtin_amdgcn_ldexpf(decode_m(j < 4 ? cm.x : cm.y, j), em - 15);
      r[j] = ev == 255 ? nan : __builtin_amdgcn_ldexpf(decode_r(j < 4 ? cv.x : cv.y, j), ev - 15);
    }
    if constexpr (kOut == 1) {
      uint32_t o[4];
      round_bf16(m, o);
      store8_bf16<kStream>(static_cast<bf16_t*>(pm), at, o);
      round_bf16(r, o);
      store8_bf16<kStream>(static_cast<bf16_t*>(pr), at, o);
    } else {
      store8<kStream>(static_cast<float*>(pm), at, m);
      store8<kStream>(static_cast<float*>(pr), at, r);
    }
  }
}

}  // namespace

hipError_t launch_square_sums(const GradTable& t, bool stream, int grid, double* parts, hipStream_t s) {
  if (stream) hipLaunchKernelGGL(square_sums_kernel<true>, dim3(grid), dim3(256), 0, s, t, parts);
  else hipLaunchKernelGGL(square_sums_kernel<false>, dim3(grid), dim3(256), 0, s, t, parts);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const double* parts, int n, double scale, double max_norm, float* out, hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(1024), 0, s, parts, n, scale, max_norm, out);
  return hipGetLastError();
}

hipError_t launch_adam(int bits, const AdamTable& t, bool stream, hipStream_t s) {
  const dim3 grid(t.chunks), block(256);
  if (bits == 8) {
    if (stream) hipLaunchKernelGGL((adam_kernel<8, true>), grid, block, 0, s, t);
    else hipLaunchKernelGGL((adam_kernel<8, false>), grid, block, 0, s, t);
  } else {
    if (stream) hipLaunchKernelGGL((adam_kernel<32, true>), grid, block, 0, s, t);
    else hipLaunchKernelGGL((adam_kernel<32, false>), grid, block, 0, s, t);
  }
  return hipGetLastError();
}

hipError_t launch_state_values(int out_dtype, const StateTable& t, bool stream, hipStream_t s) {
  const dim3 grid(t.chunks), block(256);
  if (out_dtype == 1) {
    if (stream) hipLaunchKernelGGL((state_values_kernel<1, true>), grid, block, 0, s, t);
    else hipLaunchKernelGGL((state_values_kernel<1, false>), grid, block, 0, s, t);
  } else {
    if (stream) hipLaunchKernelGGL((state_values_kernel<0, true>), grid, block, 0, s, t);
    else hipLaunchKernelGGL((state_values_kernel<0, false>), grid, block, 0, s, t);
  }
  return hipGetLastError();
}

}  // namespace moe
