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

// Four consecutive elements i .. i + 3 of a tensor of n as fp32, 0 past its end.
template <bool kStream>
__device__ __forceinline__ void load4(const void* p, bool bf16, bool aligned, int64_t i, int64_t n, float* v) {
  if (aligned && i + 4 <= n) {
    if (bf16) {
      const uint2 u = load2<kStream>(static_cast<const bf16_t*>(p) + i);
      v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    } else {
      const uint4 u = load16<kStream>(static_cast<const float*>(p) + i);
      v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
      v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = 0.0f;
      if (i + j < n)
        v[j] = bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const bf16_t*>(p)[i + j]) << 16)
                    : static_cast<const float*>(p)[i + j];
    }
  }
}

template <bool kStream>
__device__ __forceinline__ void store4(float* p, bool aligned, int64_t i, int64_t n, const float* v) {
  if (aligned && i + 4 <= n) {
    put<kStream>(p + i, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                 __float_as_uint(v[3])));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = v[j];
  }
}

// A thread's eight elements: two groups of four, from i and from i + kGap. Eight
// in a row (kGap 4) where they share a generator's call or are bf16; else 1024
// apart, so that a wave's fp32 loads and stores are whole lines.
template <int kGap, bool kStream>
__device__ __forceinline__ void load8(const void* p, bool bf16, bool aligned, int64_t i, int64_t n, float (&v)[8]) {
  if (kGap == 4 && bf16 && aligned && i + 8 <= n) {
    const uint4 u = load16<kStream>(static_cast<const bf16_t*>(p) + i);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
    return;
  }
  load4<kStream>(p, bf16, aligned, i, n, v);
  load4<kStream>(p, bf16, aligned, i + kGap, n, v + 4);
}

template <int kGap, bool kStream>
__device__ __forceinline__ void store8(float* p, bool aligned, int64_t i, int64_t n, const float (&v)[8]) {
  store4<kStream>(p, aligned, i, n, v);
  store4<kStream>(p, aligned, i + kGap, n, v + 4);
}

// w: bf16 patterns, element j in the low (even j) or high half of word j / 2
template <int kGap, bool kStream>
__device__ __forceinline__ void store8_bf16(bf16_t* p, bool aligned, int64_t i, int64_t n, const uint32_t (&w)[4]) {
  if (kGap == 4 && aligned && i + 8 <= n) {
    put<kStream>(p + i, make_uint4(w[0], w[1], w[2], w[3]));
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = i + h * kGap;
    if (aligned && at + 4 <= n) {
      put<kStream>(p + at, make_uint2(w[2 * h], w[2 * h + 1]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at + j < n) p[at + j] = static_cast<bf16_t>(w[2 * h + (j >> 1)] >> (16 * (j & 1)));
    }
  }
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
  const int e = find_tensor<kGradTensors>(t, c);
  const GradEntry& g = t.t[e];
  const void* p = g.g;
  const int64_t n = g.n;
  const bool bf16 = g.flags & 1, aligned = g.flags & 2;
  const int64_t i0 = static_cast<int64_t>(c - g.first) * t.chunk;
  double s = 0.0;
  for (int u = 0; u < t.chunk; u += 2048) {
    if (i0 + u >= n) break;
    float v[8];
    if (bf16) load8<4, kStream>(p, true, aligned, i0 + u + threadIdx.x * 8, n, v);
    else load8<1024, kStream>(p, false, aligned, i0 + u + threadIdx.x * 4, n, v);
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
__device__ __forceinline__ float decode_m(uint32_t word, int j, int e15) {
  const int c = static_cast<int>(word << (24 - 8 * (j & 3))) >> 4;
  return __builtin_amdgcn_ldexpf(__uint_as_float(static_cast<uint32_t>(c) & 0x87f00000u), e15);
}
__device__ __forceinline__ float decode_r(uint32_t word, int j, int e15) {
  return __builtin_amdgcn_ldexpf(__uint_as_float(((word >> (8 * (j & 3))) & 0xffu) << 19), e15);
}

// The scale byte of 128 elements (16 lanes of eight): the exponent whose top code
// holds the largest of them, 255 where one is not finite.
template <int kShift>
__device__ __forceinline__ int scale_of(const float (&x)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
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
    // a root above 0 stays above 0, as the update divides by it (roots of fp32 values lie above 2^-75, so their own
    // bits are past any code's; 0 leaves less than a code of u)
    t[j] = max(b, min(__float_as_uint(x[j]), 1u << 19)) << 5;
  }
  const bool bad = e == 255;
  return make_uint2(bad ? 0u : top_bytes(t[0], t[1], t[2], t[3]), bad ? 0u : top_bytes(t[4], t[5], t[6], t[7]));
}

template <bool kStream>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, bool aligned, int64_t i, int64_t n) {
  if (aligned && i + 8 <= n) return load2<kStream>(p + i);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) w[j >> 2] |= static_cast<uint32_t>(p[i + j]) << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

template <bool kStream>
__device__ __forceinline__ void store_codes(uint8_t* p, bool aligned, int64_t i, int64_t n, const uint2& c) {
  if (aligned && i + 8 <= n) {
    put<kStream>(p + i, c);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = static_cast<uint8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
}

// Square roots rounded to nearest, 0 for 0. From 2^-96 on (and for 0): the
// reciprocal root's approximation, its product with v corrected by what its
// square leaves of v. Compared with the rounded roots of every fp32 fraction in
// two binades (all there are, up to powers of 4) it gives each of them.
__device__ __forceinline__ void roots(const float (&v)[8], float (&r)[8]) {
  constexpr uint32_t kLeast = 31u << 23, kInf = 255u << 23;  // 2^-96, infinity: v is never below 0, NaN lies above
  uint32_t least = 0xffffffffu, most = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    least = min(least, __float_as_uint(v[j]) - 1u);  // (0 passes)
    most = max(most, __float_as_uint(v[j]));
  }
  if (__ballot(least < kLeast - 1u || most >= kInf) == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = __builtin_amdgcn_rsqf(__uint_as_float(max(__float_as_uint(v[j]), kLeast)));
      const float s = v[j] * y;
      r[j] = fmaf(fmaf(-s, s, v[j]), 0.5f * y, s);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = sqrtf(v[j]);
  }
}

template <int kBits, bool kStream>
__global__ __launch_bounds__(256) void adam_kernel(AdamTable t) {
#pragma clang fp contract(off)
  const uint32_t c = blockIdx.x;
  const AdamEntry& en = t.t[find_tensor<kAdamTensors>(t, c)];
  AdamScalars k = t.k;
  if (t.lr_step) adam_scalars(k, t.lr_step[0], t.lr_step[1]);
  const float gs = t.gscale ? t.gscale[0] : 1.0f;
  // gradients that are not finite as a whole: no step
  if (!(fabsf(gs) < INFINITY)) return;
  const int64_t n = en.n;
  const bool pb = en.flags & kAdamParamBf16, gb = en.flags & kAdamGradBf16, al = en.flags & kAdamAligned;
  float* master = en.master;
  const bool sr = t.stochastic && pb && !master;
  uint64_t seed = 0, offset = 0;
  if (t.rng) seed = t.rng[0], offset = t.rng[1];
  constexpr int kGap = kBits == 8 ? 4 : 1024;
  const int64_t i0 = static_cast<int64_t>(c - en.first) * t.chunk;
  for (int q = 0; q < t.chunk; q += 2048) {
    if (i0 + q >= n) break;
    const int64_t i = i0 + q + threadIdx.x * (kGap == 4 ? 8 : 4);
    float w[8], g[8], m[8], v[8];
    if (master) load8<kGap, kStream>(master, false, al, i, n, w);
    else load8<kGap, kStream>(en.p, pb, al, i, n, w);
    load8<kGap, kStream>(en.g, gb, al, i, n, g);
    float b1 = k.b1, b2 = k.b2;
    if constexpr (kBits == 32) {
      load8<kGap, kStream>(en.m, false, al, i, n, m);
      load8<kGap, kStream>(en.v, false, al, i, n, v);
    } else {
      // codes keep the ordinary way: 88 M of them stepped 177 us instead of 175, but stepped and then read out (16
      // bytes an element in all) 240 instead of 267
      const uint2 cm = load_codes<false>(static_cast<const uint8_t*>(en.m), al, i, n);
      const uint2 cv = load_codes<false>(static_cast<const uint8_t*>(en.v), al, i, n);
      const int em = i < n ? en.ms[i / kScaleBlock] : 0, ev = i < n ? en.vs[i / kScaleBlock] : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = decode_m(j < 4 ? cm.x : cm.y, j, em - 15);
        const float r = decode_r(j < 4 ? cv.x : cv.y, j, ev - 15);
        v[j] = r * r;
      }
      if (em == 255) b1 = __uint_as_float(0x7fc00000u);
      if (ev == 255) b2 = __uint_as_float(0x7fc00000u);
    }
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = g[j] * gs;
      m[j] = m[j] * b1 + x * k.c1;
      v[j] = v[j] * b2 + (x * x) * k.c2;
    }
    roots(v, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // (the reciprocal is off by 2^-23 at most, and eps keeps it in range)
      const float up = k.step_size * m[j] * __builtin_amdgcn_rcpf(fmaf(r[j], k.inv_root, k.eps));
      w[j] = w[j] - fmaf(k.decay, w[j], up);
    }
    uint32_t u[8];
    if (kBits == 8 || sr) {
      const uint64_t at = static_cast<uint64_t>(en.base + i);
      Philox x = philox(at >> 3, offset, seed);
      if constexpr (kGap != 4) {
        // each group of four is one half of a call's eight
        const Philox z = philox((at + kGap) >> 3, offset, seed);
        const bool upper = at & 4;
        x = {{upper ? x.x[2] : x.x[0], upper ? x.x[3] : x.x[1], upper ? z.x[2] : z.x[0], upper ? z.x[3] : z.x[1]}};
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[2 * j] = x.x[j] & 0xffffu;
        u[2 * j + 1] = x.x[j] >> 16;
      }
    }
    if (master) store8<kGap, kStream>(master, al, i, n, w);
    if (pb) {
      uint32_t o[4];
      if (sr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // cut after adding the number (an infinity's low bits are 0: it stays one)
          const uint32_t b = w[j] != w[j] ? 0x7fc00000u : __float_as_uint(w[j]) + u[j];
          o[j >> 1] = (j & 1) ? __builtin_amdgcn_perm(b, o[j >> 1], 0x07060302u) : b;
        }
      } else {
        round_bf16(w, o);
      }
      store8_bf16<kGap, kStream>(static_cast<bf16_t*>(en.p), al, i, n, o);
    } else {
      store8<kGap, kStream>(static_cast<float*>(en.p), al, i, n, w);
    }
    if constexpr (kBits == 32) {
      store8<kGap, kStream>(static_cast<float*>(en.m), al, i, n, m);
      store8<kGap, kStream>(static_cast<float*>(en.v), al, i, n, v);
    } else {
      // elements past the tensor's end are 0 in every row of 16 lanes
      const int em = scale_of<20>(m), ev = scale_of<19>(r);
      store_codes<false>(static_cast<uint8_t*>(en.m), al, i, n, encode_m(m, u, em));
      store_codes<false>(static_cast<uint8_t*>(en.v), al, i, n, encode_r(r, u, ev));
      if ((threadIdx.x & 15) == 0 && i < n) {
        en.ms[i / kScaleBlock] = static_cast<uint8_t>(em);
        en.vs[i / kScaleBlock] = static_cast<uint8_t>(ev);
      }
    }
  }
}

template <int kOut, bool kStream>
__global__ __launch_bounds__(256) void state_values_kernel(StateTable t) {
  const uint32_t c = blockIdx.x;
  const StateEntry& en = t.t[find_tensor<kStateTensors>(t, c)];
  const int64_t n = en.n;
  const bool al = en.aligned;
  const int64_t i0 = static_cast<int64_t>(c - en.first) * t.chunk;
  for (int q = 0; q < t.chunk; q += 2048) {
    const int64_t i = i0 + q + threadIdx.x * 8;
    if (i >= n) break;
    const uint2 cm = load_codes<kStream>(en.m, al, i, n), cv = load_codes<kStream>(en.v, al, i, n);
    const int em = en.ms[i / kScaleBlock], ev = en.vs[i / kScaleBlock];
    const float nan = __uint_as_float(0x7fc00000u);
    float m[8], r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = em == 255 ? nan : decode_m(j < 4 ? cm.x : cm.y, j, em - 15);
      r[j] = ev == 255 ? nan : decode_r(j < 4 ? cv.x : cv.y, j, ev - 15);
    }
    if constexpr (kOut == 1) {
      uint32_t o[4];
      round_bf16(m, o);
      store8_bf16<4, kStream>(static_cast<bf16_t*>(en.m_out), al, i, n, o);
      round_bf16(r, o);
      store8_bf16<4, kStream>(static_cast<bf16_t*>(en.r_out), al, i, n, o);
    } else {
      store8<4, kStream>(static_cast<float*>(en.m_out), al, i, n, m);
      store8<4, kStream>(static_cast<float*>(en.r_out), al, i, n, r);
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
