// The combine with dropout into the residual stream, and its gradient. The
// contract is in include/moe.h.
//
// The keep decisions come from a counter-based generator (Philox4x32, ten
// rounds: Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011) keyed by the seed, its counter the index of a group of
// eight consecutive elements and the caller's offset, so the backward forms the
// same decisions again and no mask is ever stored. One call yields four 32-bit
// words = eight 16-bit numbers, one per element: an element is kept when its
// number is at least thr = round(65536 p), so p is honoured to 2^-17, and kept
// values are scaled by 65536 / (65536 - thr), the reciprocal of the probability
// that is really used. Sixteen bits rather than 32 halve the generator's
// arithmetic, which would otherwise bound the backward.
#include "combine_vec.h"
#include "common.h"
#include "router.h"

namespace moe {

namespace {

struct Philox {
  uint32_t x[4];
};

__device__ __forceinline__ Philox philox(uint64_t counter, uint64_t offset, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// scale where kept, 0 where dropped, of elements 8 i .. 8 i + 7
__device__ __forceinline__ void drop8(const DropArgs& a, int64_t i, float (&f)[8]) {
  const Philox p = philox(static_cast<uint64_t>(i), a.rng[1], a.rng[0]);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = (p.x[j] & 0xffffu) >= a.thr ? a.scale : 0.0f;
    f[2 * j + 1] = (p.x[j] >> 16) >= a.thr ? a.scale : 0.0f;
  }
}

template <int kDtype>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (kDtype == 1) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[2 * i], b = reinterpret_cast<const float4*>(p)[2 * i + 1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// Stores round to nearest even and keep NaN (an fp32 to bf16 conversion instruction).
template <int kDtype>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (kDtype == 1) {
    bf16x8_t o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = static_cast<__bf16>(v[j]);
    reinterpret_cast<bf16x8_t*>(p)[i] = o;
  } else {
    reinterpret_cast<float4*>(p)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// A dropped element is the residual alone, whatever its value was (0 * inf would
// be NaN), hence a choice and not a product.
__device__ __forceinline__ float dropped(float v, float f) { return f != 0.0f ? v * f : 0.0f; }

// 256 threads of eight columns each to a (token, column band). out may be
// residual: each thread reads its elements before it writes them. Measured: 8192 x
// 6144, k 2, bf16, residual 74.7 us (403 MB, 5.4 TB/s: the rate of a large copy);
// 1500 x 1048, k 4, fp32 5.7 us. Bound by memory: each element is read once.
template <int kDtype>
__global__ __launch_bounds__(256) void combine_dropout_kernel(DropArgs a, const void* __restrict__ y,
                                                              const int32_t* __restrict__ inv_perm,
                                                              const float* __restrict__ w, const void* residual,
                                                              void* out, int64_t t0, int64_t T, int64_t d, int k,
                                                              int bands) {
  const int64_t nvec = d / 8;
  const int64_t t = t0 + blockIdx.x / bands;
  const int64_t c = static_cast<int64_t>(blockIdx.x % bands) * 256 + threadIdx.x;
  if (c >= nvec) return;
  const int64_t i = t * nvec + c;
  float acc[8], f[8], r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = 0.0f;
  if (residual) load8<kDtype>(residual, i, r);
  combine_sum<kDtype>(y, inv_perm, w, d, k, T * k, t, c, acc);
  drop8(a, i, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = dropped(acc[j], f[j]) + r[j];
  store8<kDtype>(out, i, acc);
}

// Measured: 8192 x 6144, bf16 29.3 us (201 MB, 6.9 TB/s, part of them from the
// 256 MB cache; 37 us at a large copy's rate). Bound by memory.
template <int kDtype>
__global__ __launch_bounds__(256) void dropout_backward_kernel(DropArgs a, const void* dout, void* dy, int64_t n8) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n8;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    float v[8], f[8];
    load8<kDtype>(dout, i, v);
    drop8(a, i, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = dropped(v[j], f[j]);
    store8<kDtype>(dy, i, v);
  }
}

unsigned capped(int64_t n, int64_t most) { return static_cast<unsigned>(n < most ? n : most); }

}  // namespace

hipError_t launch_combine_dropout(int dtype, const DropArgs& a, const void* y, const int32_t* inv_perm, const float* w,
                                  const void* residual, void* out, int64_t T, int64_t d, int k, hipStream_t s) {
  // 256 columns of eight to a workgroup; a launch holds fewer than 2^32 threads
  const int64_t bands = (d / 8 + 255) / 256, most = int64_t(1) << 23;
  const int64_t chunk = most > bands ? most / bands : 1;
  for (int64_t t0 = 0; t0 < T; t0 += chunk) {
    const dim3 grid(static_cast<unsigned>((T - t0 < chunk ? T - t0 : chunk) * bands));
    if (dtype == 1)
      hipLaunchKernelGGL((combine_dropout_kernel<1>), grid, dim3(256), 0, s, a, y, inv_perm, w, residual, out, t0, T, d,
                         k, static_cast<int>(bands));
    else
      hipLaunchKernelGGL((combine_dropout_kernel<0>), grid, dim3(256), 0, s, a, y, inv_perm, w, residual, out, t0, T, d,
                         k, static_cast<int>(bands));
    if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  }
  return hipSuccess;
}

hipError_t launch_dropout_backward(int dtype, const DropArgs& a, const void* dout, void* dy, int64_t T, int64_t d,
                                   hipStream_t s) {
  const int64_t n8 = T * (d / 8);
  const dim3 grid(capped((n8 + 255) / 256, int64_t(1) << 22));
  if (dtype == 1)
    hipLaunchKernelGGL((dropout_backward_kernel<1>), grid, dim3(256), 0, s, a, dout, dy, n8);
  else
    hipLaunchKernelGGL((dropout_backward_kernel<0>), grid, dim3(256), 0, s, a, dout, dy, n8);
  return hipGetLastError();
}

}  // namespace moe
