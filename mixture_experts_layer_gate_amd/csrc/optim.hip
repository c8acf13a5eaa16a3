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

// Elements i .. i + 7 of a tensor of n as fp32, 0 past its end.
__device__ __forceinline__ void load8(const void* p, bool bf16, bool aligned, int64_t i, int64_t n, float (&v)[8]) {
  if (aligned && i + 8 <= n) {
    if (bf16) {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const bf16_t*>(p) + i);
      v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
      v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
    } else {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      const float4 a = q[0], b = q[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (i + j < n)
        v[j] = bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const bf16_t*>(p)[i + j]) << 16)
                    : static_cast<const float*>(p)[i + j];
    }
  }
}

__device__ __forceinline__ void store8(float* p, bool aligned, int64_t i, int64_t n, const float (&v)[8]) {
  if (aligned && i + 8 <= n) {
    float4* q = reinterpret_cast<float4*>(p + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = v[j];
  }
}

// bits: bf16 patterns, element j in the low (even j) or high half of word j / 2
__device__ __forceinline__ void store8_bf16(bf16_t* p, bool aligned, int64_t i, int64_t n, const uint32_t (&w)[4]) {
  if (aligned && i + 8 <= n) {
    *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = static_cast<bf16_t>(w[j >> 1] >> (16 * (j & 1)));
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

__device__ __forceinline__ double chunk_squares(const GradTable& t, uint32_t c) {
  const int e = find_tensor<kGradTensors>(t, c);
  const GradEntry& g = t.t[e];
  const void* p = g.g;
  const int64_t n = g.n;
  const bool bf16 = g.bf16 & 1, aligned = !(g.bf16 & 2);
  const int64_t i0 = static_cast<int64_t>(c - g.first) * kListChunk;
  double s = 0.0;
  for (int u = threadIdx.x * 8; u < kListChunk; u += blockDim.x * 8) {
    if (i0 + u >= n) break;
    float v[8];
    load8(p, bf16, aligned, i0 + u, n, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), s);
  }
  return s;
}

__global__ __launch_bounds__(256) void square_sums_kernel(GradTable t, double* __restrict__ parts) {
  __shared__ double red[4];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) s += chunk_squares(t, c);
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

__global__ __launch_bounds__(1024) void grad_norm_small_kernel(GradTable t, double scale, double max_norm, float* out) {
  __shared__ double red[16];
  double s = 0.0;
  for (uint32_t c = 0; c < t.chunks; ++c) s += chunk_squares(t, c);
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

template <int kShift>
__device__ __forceinline__ float decode(uint32_t word, int j, int e15) {
  const uint32_t c = (word >> (8 * (j & 3))) & 0xffu;
  if constexpr (kShift == 19) {
    return __builtin_amdgcn_ldexpf(__uint_as_float(c << 19), e15);
  } else {
    const float a = __builtin_amdgcn_ldexpf(__uint_as_float((c & 0x7fu) << 20), e15);
    return __uint_as_float(__float_as_uint(a) | ((c & 0x80u) << 24));
  }
}

// The scale byte of 128 elements (16 lanes of eight): the exponent whose top code
// holds the largest of them, 255 where one is not finite.
template <int kShift>
__device__ __forceinline__ int scale_of(const float (&x)[8]) {
  int top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, static_cast<int>(__float_as_uint(x[j]) & 0x7fffffffu));
  const int e = static_cast<int>((static_cast<uint32_t>(row16_max(top)) + ((1u << kShift) - 1u)) >> 23);
  return min(e, 255);
}

// Codes of eight values: rounded by the 16-bit numbers u (up where the dropped
// bits and u reach a step).
template <int kShift>
__device__ __forceinline__ uint2 encode(const float (&x)[8], const uint32_t (&u)[8], int e) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = x[4 * h + j];
      const uint32_t bits = __float_as_uint(__builtin_amdgcn_ldexpf(fabsf(f), 15 - e));
      uint32_t c = (bits + (u[4 * h + j] << (kShift - 16))) >> kShift;
      if constexpr (kShift == 19) {
        // a root above 0 stays above 0: the update divides by it
        c = f > 0.0f ? max(c, 1u) : c;
      } else {
        c |= (__float_as_uint(f) >> 24) & 0x80u;
      }
      r |= (c & 0xffu) << (8 * j);
    }
    w[h] = e == 255 ? 0u : r;
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint2 load_codes(const uint8_t* p, bool aligned, int64_t i, int64_t n) {
  if (aligned && i + 8 <= n) return *reinterpret_cast<const uint2*>(p + i);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) w[j >> 2] |= static_cast<uint32_t>(p[i + j]) << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(uint8_t* p, bool aligned, int64_t i, int64_t n, const uint2& c) {
  if (aligned && i + 8 <= n) {
    *reinterpret_cast<uint2*>(p + i) = c;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = static_cast<uint8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
}

template <int kBits>
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
  const int64_t i0 = static_cast<int64_t>(c - en.first) * kListChunk;
  for (int q = 0; q < kListChunk; q += 2048) {
    if (i0 + q >= n) break;
    const int64_t i = i0 + q + threadIdx.x * 8;
    float w[8], g[8], m[8], v[8];
    if (master) load8(master, false, al, i, n, w);
    else load8(en.p, pb, al, i, n, w);
    load8(en.g, gb, al, i, n, g);
    float b1 = k.b1, b2 = k.b2;
    if constexpr (kBits == 32) {
      load8(en.m, false, al, i, n, m);
      load8(en.v, false, al, i, n, v);
    } else {
      const uint2 cm = load_codes(static_cast<const uint8_t*>(en.m), al, i, n);
      const uint2 cv = load_codes(static_cast<const uint8_t*>(en.v), al, i, n);
      const int em = i < n ? en.ms[i / kScaleBlock] : 0, ev = i < n ? en.vs[i / kScaleBlock] : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = decode<20>(j < 4 ? cm.x : cm.y, j, em - 15);
        const float r = decode<19>(j < 4 ? cv.x : cv.y, j, ev - 15);
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
      r[j] = sqrtf(v[j]);
      const float up = (k.step_size * m[j]) / (r[j] * k.inv_root + k.eps);
      w[j] = w[j] - (up + k.decay * w[j]);
    }
    uint32_t u[8];
    if (kBits == 8 || sr) {
      const Philox x = philox(static_cast<uint64_t>(en.base + i) >> 3, offset, seed);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[2 * j] = x.x[j] & 0xffffu;
        u[2 * j + 1] = x.x[j] >> 16;
      }
    }
    if (master) store8(master, al, i, n, w);
    if (pb) {
      uint32_t o[4];
      if (sr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t h[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t bits = __float_as_uint(w[2 * j + z]);
            // infinities and NaN stay what they are
            h[z] = (bits & 0x7f800000u) == 0x7f800000u ? bits | ((bits & 0xffffu) ? 0x400000u : 0u)
                                                       : bits + u[2 * j + z];
          }
          o[j] = (h[0] >> 16) | (h[1] & 0xffff0000u);
        }
      } else {
        round_bf16(w, o);
      }
      store8_bf16(static_cast<bf16_t*>(en.p), al, i, n, o);
    } else {
      store8(static_cast<float*>(en.p), al, i, n, w);
    }
    if constexpr (kBits == 32) {
      store8(static_cast<float*>(en.m), al, i, n, m);
      store8(static_cast<float*>(en.v), al, i, n, v);
    } else {
      // elements past the tensor's end are 0 in every row of 16 lanes
      const int em = scale_of<20>(m), ev = scale_of<19>(r);
      store_codes(static_cast<uint8_t*>(en.m), al, i, n, encode<20>(m, u, em));
      store_codes(static_cast<uint8_t*>(en.v), al, i, n, encode<19>(r, u, ev));
      if ((threadIdx.x & 15) == 0 && i < n) {
        en.ms[i / kScaleBlock] = static_cast<uint8_t>(em);
        en.vs[i / kScaleBlock] = static_cast<uint8_t>(ev);
      }
    }
  }
}

template <int kOut>
__global__ __launch_bounds__(256) void state_values_kernel(StateTable t) {
  const uint32_t c = blockIdx.x;
  const StateEntry& en = t.t[find_tensor<kStateTensors>(t, c)];
  const int64_t n = en.n;
  const bool al = en.aligned;
  const int64_t i0 = static_cast<int64_t>(c - en.first) * kListChunk;
  for (int q = 0; q < kListChunk; q += 2048) {
    const int64_t i = i0 + q + threadIdx.x * 8;
    if (i >= n) break;
    const uint2 cm = load_codes(en.m, al, i, n), cv = load_codes(en.v, al, i, n);
    const int em = en.ms[i / kScaleBlock], ev = en.vs[i / kScaleBlock];
    const float nan = __uint_as_float(0x7fc00000u);
    float m[8], r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = em == 255 ? nan : decode<20>(j < 4 ? cm.x : cm.y, j, em - 15);
      r[j] = ev == 255 ? nan : decode<19>(j < 4 ? cv.x : cv.y, j, ev - 15);
    }
    if constexpr (kOut == 1) {
      uint32_t o[4];
      round_bf16(m, o);
      store8_bf16(static_cast<bf16_t*>(en.m_out), al, i, n, o);
      round_bf16(r, o);
      store8_bf16(static_cast<bf16_t*>(en.r_out), al, i, n, o);
    } else {
      store8(static_cast<float*>(en.m_out), al, i, n, m);
      store8(static_cast<float*>(en.r_out), al, i, n, r);
    }
  }
}

}  // namespace

hipError_t launch_square_sums(const GradTable& t, int grid, double* parts, hipStream_t s) {
  hipLaunchKernelGGL(square_sums_kernel, dim3(grid), dim3(256), 0, s, t, parts);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const double* parts, int n, double scale, double max_norm, float* out, hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(1024), 0, s, parts, n, scale, max_norm, out);
  return hipGetLastError();
}

hipError_t launch_grad_norm_small(const GradTable& t, double scale, double max_norm, float* out, hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_small_kernel, dim3(1), dim3(1024), 0, s, t, scale, max_norm, out);
  return hipGetLastError();
}

hipError_t launch_adam(int bits, const AdamTable& t, hipStream_t s) {
  if (bits == 8) hipLaunchKernelGGL(adam_kernel<8>, dim3(t.chunks), dim3(256), 0, s, t);
  else hipLaunchKernelGGL(adam_kernel<32>, dim3(t.chunks), dim3(256), 0, s, t);
  return hipGetLastError();
}

hipError_t launch_state_values(int out_dtype, const StateTable& t, hipStream_t s) {
  if (out_dtype == 1) hipLaunchKernelGGL(state_values_kernel<1>, dim3(t.chunks), dim3(256), 0, s, t);
  else hipLaunchKernelGGL(state_values_kernel<0>, dim3(t.chunks), dim3(256), 0, s, t);
  return hipGetLastError();
}

}  // namespace moe
