// The norm in front of the layer (RMS or layer norm, the residual added) and its
// gradients. The contract is in include/moe.h.
#include "common.h"
#include "train.h"

namespace moe {

namespace {

// One 16-byte vector of a row: eight bf16 or four fp32 values.
template <int kDtype> constexpr int kVec = kDtype == 1 ? 8 : 4;

template <int kDtype>
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[kVec<kDtype>]) {
  if constexpr (kDtype == 1) {
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  } else {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  }
}

// Rounds to nearest even and keeps NaN (an fp32 to bf16 conversion instruction).
template <int kDtype>
__device__ __forceinline__ uint4 pack(const float (&v)[kVec<kDtype>]) {
  if constexpr (kDtype == 1) {
    bf16x8_t o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = static_cast<__bf16>(v[j]);
    return *reinterpret_cast<uint4*>(&o);
  } else {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
}

// Elements N i .. N i + N - 1 of a weight vector of either type.
template <int N>
__device__ __forceinline__ void load_w(const void* p, int w_bf16, int i, float (&v)[N]) {
  if (w_bf16) {
    if constexpr (N == 8) {
      unpack<1>(reinterpret_cast<const uint4*>(p)[i], v);
    } else {
      const uint2 u = reinterpret_cast<const uint2*>(p)[i];
      v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    }
  } else {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const float4 a = reinterpret_cast<const float4*>(p)[i * (N / 4) + q];
      v[4 * q] = a.x; v[4 * q + 1] = a.y; v[4 * q + 2] = a.z; v[4 * q + 3] = a.w;
    }
  }
}

// kStream: a batch of over half the 256 MB cache passes through once, and no cache
// line is kept for what it reads, nor for the sum, which the backward reads much
// later; y and dx stay in it for what runs next. Measured, ordinary loads and
// stores, these, and y and dx streaming too: norm of 16384 x 6144 with residual
// alone 153, 152 and 145 us, but with a gate of 8 experts behind it 218, 204 and
// 214; gradients of 8192 x 6144 with the next layer's dropout 109, 100 and 109;
// norm of 4096 x 7168 alone 45, 40 and 41, with the gate 84, 75 and 85. Gradients
// of 2047 x 6144 with bias, which the cache holds: 22 us, and 24 with streaming.
template <bool kStream>
__device__ __forceinline__ uint4 get(const uint4* p) {
  const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p);
  const u32x4_t v = kStream ? __builtin_nontemporal_load(q) : *q;
  return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool kStream>
__device__ __forceinline__ void put(uint4* p, const uint4& v) {
  u32x4_t* q = reinterpret_cast<u32x4_t*>(p);
  if (kStream) __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, q);
  else *q = u32x4_t{v.x, v.y, v.z, v.w};
}

// Sum over a wave in every lane: rows of 16 by rotations inside them, then the
// four rows' sums.
template <int kRor>
__device__ __forceinline__ float ror_add(float v) {
  return v + __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), 0x120 + kRor, 0xf, 0xf, false));
}
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = ror_add<1>(ror_add<2>(ror_add<4>(ror_add<8>(v))));
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

__device__ __forceinline__ float sum4(const float4& v) { return (v.x + v.y) + (v.z + v.w); }

__device__ __forceinline__ float sum16(const float* p) {
  const float4* q = reinterpret_cast<const float4*>(p);
  return (sum4(q[0]) + sum4(q[1])) + (sum4(q[2]) + sum4(q[3]));
}

// Sums over the workgroup (kWaveRow: over the wave), the same values in every
// thread, by one exchange. red: one float to a wave, 16 of them for each sum, those
// without a wave 0.
template <bool kWaveRow, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[16]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
  if constexpr (kWaveRow) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[k][threadIdx.x >> 6] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = sum16(red[k]);
}

constexpr float kShrink = 0x1p-80f;

// One row to a workgroup (kWaveRow: to a wave), kept in registers as fp32: NV
// vectors to a thread. The variance is that of the differences to the mean, taken
// from the registers, and the same exchange gives what the mean's own rounding lost,
// so rows whose mean is many times their spread keep their precision (16384 x 7168
// in bf16 with a residual, written to the same outputs again: 147.5 us, and 145.8
// without that). A row whose sums pass fp32's range is scaled by 2^-80 and summed
// again, so the statistics are right for every finite row.
template <int kDtype, bool kLayer, int NV, bool kWaveRow, bool kStream>
__global__ __launch_bounds__(kWaveRow ? 256 : 1024) void norm_kernel(NormArgs a) {
  constexpr int V = kVec<kDtype>;
  __shared__ __attribute__((aligned(16))) float red[3][16];
  if (!kWaveRow && threadIdx.x < 48) red[threadIdx.x >> 4][threadIdx.x & 15] = 0.0f;
  if (!kWaveRow) __syncthreads();
  const int nvec = a.d / V;
  const int lanes = kWaveRow ? 64 : blockDim.x;
  const int tid = kWaveRow ? (threadIdx.x & 63) : threadIdx.x;
  const int per = kWaveRow ? (blockDim.x >> 6) : 1;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  uint4 ux[NV], ur[NV];
  const auto fetch = [&](int64_t t) {
    const uint4* px = reinterpret_cast<const uint4*>(a.x) + t * nvec;
    const uint4* pr = reinterpret_cast<const uint4*>(a.residual) + t * nvec;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * lanes;
      ux[j] = c < nvec ? get<kStream>(px + c) : make_uint4(0, 0, 0, 0);
      if (a.residual) ur[j] = c < nvec ? get<kStream>(pr + c) : make_uint4(0, 0, 0, 0);
    }
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * per + (kWaveRow ? (threadIdx.x >> 6) : 0);
  if (t < a.T) fetch(t);
  float w[NV][V], b[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = tid + j * lanes;
    if (a.w && c < nvec) load_w<V>(a.w, a.w_bf16, c, w[j]);
    if (kLayer && a.b && c < nvec) load_w<V>(a.b, a.w_bf16, c, b[j]);
  }
  for (; t < a.T; t += step) {
    float v[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * lanes;
      unpack<kDtype>(ux[j], v[j]);
      uint4 o = ux[j];
      if (a.residual) {
        float r[V];
        unpack<kDtype>(ur[j], r);
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] += r[i];
        o = pack<kDtype>(v[j]);
        unpack<kDtype>(o, v[j]);
      }
      if (a.sum && c < nvec) put<kStream>(reinterpret_cast<uint4*>(a.sum) + t * nvec + c, o);
    }
    // the next row is on its way while this one's sums are exchanged
    if (t + step < a.T) fetch(t + step);
    // mean + rest is the mean: rest, the mean of the differences to the first one, is
    // what that sum's rounding lost of it
    float mean = 0.0f, rest = 0.0f, var = 0.0f;
    bool small = false;  // scaled by kShrink
    for (;;) {
      if constexpr (kLayer) {
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) s[0] += v[j][i];
        row_sums<kWaveRow>(s, red);
        mean = s[0] * inv_d;
      }
      float q[kLayer ? 2 : 1] = {};
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (tid + j * lanes < nvec) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float e = kLayer ? v[j][i] - mean : v[j][i];
            q[0] = fmaf(e, e, q[0]);
            if constexpr (kLayer) q[1] += e;
          }
        }
      row_sums<kWaveRow>(q, red + 1);
      var = q[0] * inv_d;
      if constexpr (kLayer) {
        rest = q[1] * inv_d;
        var = fmaf(-rest, rest, var);
        var = var < 0.0f ? 0.0f : var;  // (NaN stays)
      }
      if (small || var < INFINITY) break;
      small = true;
      if (!kWaveRow) __syncthreads();  // red is written again
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] *= kShrink;
    }
    // (a row with an infinity: the mean is that infinity, rest NaN)
    float rstd, mul, mean_out = fabsf(mean) == INFINITY ? mean : mean + rest;
    if (!small) {
      rstd = mul = 1.0f / sqrtf(var + a.eps);
    } else {
      const double up = 1.0 / static_cast<double>(kShrink);
      const double r = 1.0 / sqrt(static_cast<double>(var) * up * up + static_cast<double>(a.eps));
      rstd = static_cast<float>(r);
      mul = r * up > 0x1.fffffep127 ? 0x1.fffffep127f : static_cast<float>(r * up);  // (NaN stays)
      mean_out = static_cast<float>(static_cast<double>(mean_out) * up);
    }
    const float shift = -rest * mul;
    if (tid == 0) {
      if (kLayer && a.mean) a.mean[t] = mean_out;
      if (a.rstd) a.rstd[t] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * lanes;
      if (c >= nvec) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float y = kLayer ? fmaf(v[j][i] - mean, mul, shift) : v[j][i] * mul;
        if (a.w) y *= w[j][i];
        if (kLayer && a.b) y += b[j][i];
        v[j][i] = y;
      }
      reinterpret_cast<uint4*>(a.y)[t * nvec + c] = pack<kDtype>(v[j]);
    }
    // red is written again; alternating parts of it without this barrier let the waves
    // drift apart (16384 x 7168, layer norm with a residual: 145 and 165 us; RMS norm equal)
    if (!kWaveRow) __syncthreads();
  }
}

template <int kDtype, int NV, bool kWaveRow>
constexpr bool wide() {
  return !kWaveRow && NV * kVec<kDtype> > 8;
}

// A layer norm's row so far from zero that the rounding of its mean is looked after in
// the gradients: within 8 spreads it puts h off by at most 2^-21. (A NaN row is NaN
// either way.)
constexpr float kFar = 8.0f;
__device__ __forceinline__ bool far_row(float mean, float rstd) { return fabsf(mean * rstd) > kFar; }

// Gradients: with h = (x - mean) rstd and g = dy w,
//   dx = rstd (g - mean(g) - h mean(g h)) + dx_in      (mean(g): layer norm)
//   dw = sum_t dy h,  db = sum_t dy.
// A workgroup takes every parts-th row and keeps its columns' sums of dw and db
// in registers; the parts are summed by norm_parts_kernel in their order. Both
// row means come from one exchange between the waves.
// Layer norm: the mean that is handed in is rounded, which puts every h of a row off
// by one amount, its rounding times rstd (3 % of the spread for unit spread around
// 10^6 in fp32). The mean of h is that amount, and in rows far from zero it is taken
// back before h is used.
// Differences to the mean are formed at half size and rstd at double, so that
// neither passes fp32's range where h does not.
template <int kDtype, bool kLayer, int NV, bool kWaveRow, bool kStream, bool kSums>
__device__ __forceinline__ void grad_rows(const NormGradArgs& a, int block, int blocks) {
  constexpr int V = kVec<kDtype>;
  __shared__ __attribute__((aligned(16))) float red[2][3][16];
  if (!kWaveRow) {
    // (rows to workgroups have 192 threads and more)
    if (threadIdx.x < 96) (&red[0][0][0])[threadIdx.x] = 0.0f;
    __syncthreads();
  }
  const int nvec = a.d / V;
  const int lanes = kWaveRow ? 64 : blockDim.x;
  const int tid = kWaveRow ? (threadIdx.x & 63) : threadIdx.x;
  const int nw = blockDim.x >> 6;
  const int per = kWaveRow ? nw : 1;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const int64_t step = static_cast<int64_t>(blocks) * per;
  // 16 columns to a thread of a full workgroup leave no registers for their sums, for
  // the next row and for the weights, which are read again for every row then
  constexpr bool kWide = wide<kDtype, NV, kWaveRow>();
  static_assert(!(kWide && kSums), "columns summed apart");
  float aw[NV][V], ab[NV][V], w[kWide ? 1 : NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      aw[j][i] = ab[j][i] = 0.0f;
      if (!kWide) w[j][i] = 1.0f;
    }
    if (!kWide && a.w && tid + j * lanes < nvec) load_w<V>(a.w, a.w_bf16, tid + j * lanes, w[j]);
  }
  uint4 ud[NV], ux[NV], ui[NV];
  float rstd = 0.0f, mean = 0.0f;
  const auto fetch = [&](int64_t t) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * lanes;
      const bool in = c < nvec;
      const int64_t at = t * nvec + c;
      ud[j] = in ? get<kStream>(reinterpret_cast<const uint4*>(a.dy) + at) : make_uint4(0, 0, 0, 0);
      ux[j] = in ? get<kStream>(reinterpret_cast<const uint4*>(a.x) + at) : make_uint4(0, 0, 0, 0);
      if (!kWide && a.dx_in)
        ui[j] = in ? get<kStream>(reinterpret_cast<const uint4*>(a.dx_in) + at) : make_uint4(0, 0, 0, 0);
    }
    rstd = a.rstd[t];
    if constexpr (kLayer) mean = a.mean[t];
  };
  int64_t t = static_cast<int64_t>(block) * per + (kWaveRow ? (threadIdx.x >> 6) : 0);
  if (!kWide && t < a.T) fetch(t);
  for (int half = 0; t < a.T; t += step, half ^= 1) {
    if (kWide) fetch(t);
    const float rs = rstd, r2 = 2.0f * rstd, m2 = kLayer ? -0.5f * mean : 0.0f;
    float h[NV][V], g[NV][V];
    uint4 add[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack<kDtype>(ux[j], h[j]);
      unpack<kDtype>(ud[j], g[j]);
      if (!kWide) add[j] = ui[j];
    }
    // the next row is on its way while this one's sums are exchanged
    if (!kWide && t + step < a.T) fetch(t + step);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) h[j][i] = tid + j * lanes < nvec ? fmaf(h[j][i], 0.5f, m2) * r2 : 0.0f;
    if (kLayer && far_row(m2, r2)) {
      float c = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) c += h[j][i];
      c = wave_sum(c);
      if constexpr (!kWaveRow) {
        if ((threadIdx.x & 63) == 0) red[half][2][threadIdx.x >> 6] = c;
        __syncthreads();
        c = sum16(red[half][2]);
      }
      c *= inv_d;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) h[j][i] = tid + j * lanes < nvec ? h[j][i] - c : 0.0f;
    }
    float sg = 0.0f, sh = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = tid + j * lanes < nvec;
      if constexpr (kWide) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[0][i] = 1.0f;
        if (a.w && in) load_w<V>(a.w, a.w_bf16, tid + j * lanes, w[0]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (kSums) aw[j][i] = fmaf(g[j][i], h[j][i], aw[j][i]);
        if constexpr (kSums && kLayer) ab[j][i] += g[j][i];
        g[j][i] *= w[kWide ? 0 : j][i];
        if constexpr (kLayer) sg += g[j][i];
        sh = fmaf(g[j][i], h[j][i], sh);
      }
    }
    if constexpr (kLayer) sg = wave_sum(sg);
    sh = wave_sum(sh);
    if constexpr (!kWaveRow) {
      // (the other half is read until every wave is past this barrier)
      if ((threadIdx.x & 63) == 0) {
        red[half][0][threadIdx.x >> 6] = sh;
        if (kLayer) red[half][1][threadIdx.x >> 6] = sg;
      }
      __syncthreads();
      sh = sum16(red[half][0]);
      if constexpr (kLayer) sg = sum16(red[half][1]);
    }
    sg *= inv_d;
    sh *= inv_d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * lanes;
      if (c >= nvec) continue;
      float o[V];
      if (kWide && a.dx_in) add[j] = reinterpret_cast<const uint4*>(a.dx_in)[t * nvec + c];
      if (a.dx_in) unpack<kDtype>(add[j], o);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float e = fmaf(-h[j][i], sh, g[j][i]);
        if constexpr (kLayer) e -= sg;
        o[i] = a.dx_in ? fmaf(e, rs, o[i]) : e * rs;
      }
      reinterpret_cast<uint4*>(a.dx)[t * nvec + c] = pack<kDtype>(o);
    }
  }
  if constexpr (!kSums) return;
  // this workgroup's part
  if constexpr (kWaveRow) {
    __shared__ float joined[64 * NV * V];
    for (int which = 0; which < (kLayer ? 2 : 1); ++which) {
      float* part = which == 0 ? a.part_w : a.part_b;
      if (!part) continue;
      for (int k = 0; k < nw; ++k) {
        __syncthreads();
        if ((threadIdx.x >> 6) == k) {
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              float* p = joined + (j * V + i) * 64 + tid;
              const float v = which == 0 ? aw[j][i] : ab[j][i];
              *p = k == 0 ? v : *p + v;
            }
        }
      }
      if ((threadIdx.x >> 6) == nw - 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = tid + j * 64;
          if (c >= nvec) continue;
          float4* p = reinterpret_cast<float4*>(part + static_cast<int64_t>(block) * a.d + c * V);
#pragma unroll
          for (int q = 0; q < V / 4; ++q) {
            const float* f = joined + (j * V + 4 * q) * 64 + tid;
            p[q] = make_float4(f[0], f[64], f[128], f[192]);
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * lanes;
      if (c >= nvec) continue;
      const int64_t at = static_cast<int64_t>(block) * a.d + c * V;
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        if (a.part_w)
          reinterpret_cast<float4*>(a.part_w + at)[q] =
              make_float4(aw[j][4 * q], aw[j][4 * q + 1], aw[j][4 * q + 2], aw[j][4 * q + 3]);
        if (kLayer && a.part_b)
          reinterpret_cast<float4*>(a.part_b + at)[q] =
              make_float4(ab[j][4 * q], ab[j][4 * q + 1], ab[j][4 * q + 2], ab[j][4 * q + 3]);
      }
    }
  }
}

template <int kDtype, bool kLayer, int NV, bool kWaveRow, bool kStream>
__global__ __launch_bounds__(kWaveRow ? 256 : 1024) void norm_grad_kernel(NormGradArgs a) {
  grad_rows<kDtype, kLayer, NV, kWaveRow, kStream, true>(a, blockIdx.x, gridDim.x);
}

// The means of the h of N rows of a layer norm, what the rounding of the rows' means put
// them off by: all rows by one wave, the same values in every lane.
template <int kDtype, int N>
__device__ __forceinline__ void shifts_of(const NormGradArgs& a, const int64_t (&t)[N], float (&c)[N]) {
  constexpr int V = kVec<kDtype>;
  const int nvec = a.d / V;
  float r2[N], m2[N];
  double s[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    r2[n] = 2.0f * a.rstd[t[n]];
    m2[n] = -0.5f * a.mean[t[n]];
    s[n] = 0.0;
  }
#pragma unroll 2
  for (int k = threadIdx.x & 63; k < nvec; k += 64) {
    uint4 u[N];
#pragma unroll
    for (int n = 0; n < N; ++n) u[n] = reinterpret_cast<const uint4*>(a.x)[t[n] * nvec + k];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float h[V], e = 0.0f;
      unpack<kDtype>(u[n], h);
#pragma unroll
      for (int i = 0; i < V; ++i) e += fmaf(h[i], 0.5f, m2[n]) * r2[n];
      s[n] += e;
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s[n] += __shfl_xor(s[n], o);
    c[n] = static_cast<float>(s[n] / a.d);
  }
}

// Those means of the rows that are far from zero; the others are not read, nor theirs
// written.
template <int kDtype>
__global__ __launch_bounds__(256) void norm_shift_kernel(NormGradArgs a) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 4;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); t < a.T; t += step) {
    if (!far_row(a.mean[t], a.rstd[t])) continue;
    const int64_t row[1] = {t};
    float c[1];
    shifts_of<kDtype>(a, row, c);
    if ((threadIdx.x & 63) == 0) a.shift[t] = c[0];
  }
}

// dw and db of 64 bytes of columns over all rows, which need nothing but the rows'
// statistics: four vectors to a row, a row to every four threads. A thread's sums
// go into its total every 32 rows; the threads' totals are joined inside the rows
// of 16 lanes, then between those, in a fixed order.
// Layer norm: rows far from zero are left out of dw, and a wave that has met some adds
// them once it knows what their h are off by. For rows over 8192 columns a launch in front has formed it (2047 x 16384
// in bf16 74 us without that launch, 76 with it, 123 where every row is far); shorter
// ones are read again by the wave, which costs other batches next to nothing (333 x 1048
// in fp32 3.6 and 3.8 us, 700 x 7168 in bf16 18.1 and 18.4, but 42 and 132 where every
// row is far).
template <int kDtype, bool kLayer>
__device__ __forceinline__ void grad_columns(const NormGradArgs& a, int block, float* dw, float* db) {
  constexpr int V = kVec<kDtype>;
  __shared__ float join[kLayer ? 2 : 1][64][4 * V];
  const int nvec = a.d / V, groups = blockDim.x >> 2;
  const int q = threadIdx.x & 3, c = block * 4 + q;
  float tw[V], tb[V];
#pragma unroll
  for (int i = 0; i < V; ++i) tw[i] = tb[i] = 0.0f;
  float most = 0.0f;  // the farthest of this thread's rows, in spreads
  if (c < nvec) {
    for (int64_t t0 = threadIdx.x >> 2; t0 < a.T; t0 += 32 * groups) {
      const int64_t end = t0 + 32 * groups < a.T ? t0 + 32 * groups : a.T;
      float aw[V], ab[V];
#pragma unroll
      for (int i = 0; i < V; ++i) aw[i] = ab[i] = 0.0f;
#pragma unroll 4
      for (int64_t t = t0; t < end; t += groups) {
        const int64_t at = t * nvec + c;
        float g[V], h[V];
        unpack<kDtype>(reinterpret_cast<const uint4*>(a.dy)[at], g);
        unpack<kDtype>(reinterpret_cast<const uint4*>(a.x)[at], h);
        const float r2 = 2.0f * a.rstd[t], m2 = kLayer ? -0.5f * a.mean[t] : 0.0f;
        const bool later = kLayer && far_row(m2, r2);
        if constexpr (kLayer) most = fmaxf(most, fabsf(m2 * r2));
#pragma unroll
        for (int i = 0; i < V; ++i) {
          aw[i] = fmaf(later ? 0.0f : g[i], fmaf(h[i], 0.5f, m2) * r2, aw[i]);
          if constexpr (kLayer) ab[i] += g[i];
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        tw[i] += aw[i];
        tb[i] += ab[i];
      }
    }
  }
  if (kLayer && dw && __ballot(most > kFar)) {
    // 16 rows of the wave at a time, each taken in by its four lanes
    const int mine = (threadIdx.x & 63) >> 2;
    for (int64_t t0 = 16 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); t0 < a.T; t0 += groups) {
      const int64_t t = t0 + mine;
      const bool at = t < a.T && far_row(a.mean[t], a.rstd[t]);
      float off = 0.0f;
      if (a.shift) {
        if (at) off = a.shift[t];
      } else {
        for (uint64_t left = __ballot(at); left;) {
          // four rows at once (fewer: the last one again), so that their loads overlap
          int k[4];
          int64_t rows[4];
          float m[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            k[n] = left ? __builtin_ctzll(left) >> 2 : k[n > 0 ? n - 1 : 0];
            rows[n] = t0 + k[n];
            left &= ~(15ull << (4 * k[n]));
          }
          shifts_of<kDtype>(a, rows, m);
#pragma unroll
          for (int n = 0; n < 4; ++n)
            if (mine == k[n]) off = m[n];
        }
      }
      if (at && c < nvec) {
        float g[V], h[V];
        unpack<kDtype>(reinterpret_cast<const uint4*>(a.dy)[t * nvec + c], g);
        unpack<kDtype>(reinterpret_cast<const uint4*>(a.x)[t * nvec + c], h);
        const float r2 = 2.0f * a.rstd[t], m2 = -0.5f * a.mean[t];
#pragma unroll
        for (int i = 0; i < V; ++i) tw[i] = fmaf(g[i], fmaf(h[i], 0.5f, m2) * r2 - off, tw[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    tw[i] = ror_add<4>(ror_add<8>(tw[i]));
    if constexpr (kLayer) tb[i] = ror_add<4>(ror_add<8>(tb[i]));
  }
  if ((threadIdx.x & 15) < 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      join[0][threadIdx.x >> 4][q * V + i] = tw[i];
      if constexpr (kLayer) join[kLayer ? 1 : 0][threadIdx.x >> 4][q * V + i] = tb[i];
    }
  }
  __syncthreads();
  const int which = threadIdx.x / (4 * V), i = threadIdx.x % (4 * V), col = block * 4 * V + i;
  if (which < (kLayer ? 2 : 1) && col < a.d) {
    float* out = which == 0 ? dw : db;
    if (out) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // (a multiple of four rows of 16 lanes: whole waves)
      for (unsigned r = 0; r < blockDim.x >> 4; r += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] += join[which][r + k][i];
      }
      out[col] = (s[0] + s[1]) + (s[2] + s[3]);
    }
  }
}

// Both in one launch: the first `columns` workgroups sum dw and db, the others form
// dx. For short batches, where reading dy and x twice costs less than writing parts
// and a launch to sum them, and for rows of over 8192 columns, whose sums leave a
// thread no registers (2047 x 16384 with bias: 94 us, and 644 with parts). Measured against
// parts: 32 x 7168 4.3 and 7.0 us, 512 x 7168 12.3 and 15.4, 768 x 7168 17.0 and
// 15.6; 1024 x 4096 with bias 12.5 and 15.2, 2047 x 4096 21.7 and 20.3; 1024 x 512
// 4.9 and 7.3, 2047 x 512 12.4 and 8.0.
template <int kDtype, bool kLayer, int NV, bool kWaveRow>
__global__ __launch_bounds__(kWaveRow ? 256 : 1024) void norm_grad_short_kernel(NormGradArgs a, int columns, float* dw,
                                                                                float* db) {
  if (static_cast<int>(blockIdx.x) < columns) grad_columns<kDtype, kLayer>(a, blockIdx.x, dw, db);
  else grad_rows<kDtype, kLayer, NV, kWaveRow, false, false>(a, blockIdx.x - columns, gridDim.x - columns);
}

// Column sums of the parts: 16 columns to a workgroup (64 bytes of a part's row),
// four to a thread; its threads' sums are joined inside the waves, then between
// them, in a fixed order. 256 threads up to 256 parts, 1024 above (measured at
// 512 parts of 512 columns: 12.4 and 11.3 us with the rows' pass of 8192; at 256
// parts of 7168 columns 42.4 and 42.9 with that of 4096).
__global__ __launch_bounds__(1024) void norm_parts_kernel(const float* __restrict__ part_w,
                                                          const float* __restrict__ part_b, int parts, int d,
                                                          float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float4 join[16][4];
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;
  const int q = threadIdx.x & 3, groups = blockDim.x >> 2;
  const int c = blockIdx.x * 16 + q * 4;
  float4 s = make_float4(0, 0, 0, 0);
  if (c < d) {
    for (int p = threadIdx.x >> 2; p < parts; p += groups) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(p) * d + c);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
#pragma unroll
  for (int o = 4; o < 64; o <<= 1) {
    s.x += __shfl_xor(s.x, o);
    s.y += __shfl_xor(s.y, o);
    s.z += __shfl_xor(s.z, o);
    s.w += __shfl_xor(s.w, o);
  }
  if ((threadIdx.x & 63) < 4) join[threadIdx.x >> 6][q] = s;
  __syncthreads();
  if (threadIdx.x < 4 && c < d) {
    for (unsigned i = 1; i < blockDim.x >> 6; ++i) {
      const float4 v = join[i][q];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    *reinterpret_cast<float4*>(out + c) = s;
  }
}

struct Shape {
  bool wave;    // one row to a wave
  int nv;       // vectors to a thread
  int threads;
};

Shape row_shape(int dtype, int64_t d, int most) {
  const int64_t nvec = d / (dtype == 1 ? 8 : 4);
  // rows of at most 128 vectors: a wave to each, four to a workgroup
  if (nvec <= 64) return {true, 1, 256};
  if (nvec <= 128) return {true, 2, 256};
  int nv = 1;
  while (nvec > static_cast<int64_t>(most) * nv && nv < 4) nv *= 2;
  return {false, nv, static_cast<int>((nvec + 64 * nv - 1) / (64 * nv)) * 64};
}

// The kernel of a shape: Fn::launch<dtype, layer, NV, wave, stream>.
template <int kDtype, bool kLayer, bool kStream, typename Fn>
void by_shape(const Shape& sh, const Fn& f) {
  if (sh.wave) {
    if (sh.nv == 1) f.template launch<kDtype, kLayer, 1, true, kStream>();
    else f.template launch<kDtype, kLayer, 2, true, kStream>();
  } else if (sh.nv == 1) {
    f.template launch<kDtype, kLayer, 1, false, kStream>();
  } else if (sh.nv == 2) {
    f.template launch<kDtype, kLayer, 2, false, kStream>();
  } else if constexpr (kDtype == 0) {
    f.template launch<kDtype, kLayer, 4, false, kStream>();
  }
}
template <typename Fn>
void by_type(int dtype, bool layer, bool stream, const Shape& sh, const Fn& f) {
  if (dtype == 1) {
    if (stream) layer ? by_shape<1, true, true>(sh, f) : by_shape<1, false, true>(sh, f);
    else layer ? by_shape<1, true, false>(sh, f) : by_shape<1, false, false>(sh, f);
  } else {
    if (stream) layer ? by_shape<0, true, true>(sh, f) : by_shape<0, false, true>(sh, f);
    else layer ? by_shape<0, true, false>(sh, f) : by_shape<0, false, false>(sh, f);
  }
}

struct NormLaunch {
  const NormArgs& a;
  dim3 grid, block;
  hipStream_t s;
  template <int kDtype, bool kLayer, int NV, bool kWaveRow, bool kStream>
  void launch() const {
    hipLaunchKernelGGL((norm_kernel<kDtype, kLayer, NV, kWaveRow, kStream>), grid, block, 0, s, a);
  }
};
struct NormGradLaunch {
  const NormGradArgs& a;
  dim3 grid, block;
  hipStream_t s;
  template <int kDtype, bool kLayer, int NV, bool kWaveRow, bool kStream>
  void launch() const {
    if constexpr (!wide<kDtype, NV, kWaveRow>())
      hipLaunchKernelGGL((norm_grad_kernel<kDtype, kLayer, NV, kWaveRow, kStream>), grid, block, 0, s, a);
  }
};

struct NormShortLaunch {
  const NormGradArgs& a;
  int columns;
  float *dw, *db;
  dim3 grid, block;
  hipStream_t s;
  template <int kDtype, bool kLayer, int NV, bool kWaveRow, bool kStream>
  void launch() const {
    hipLaunchKernelGGL((norm_grad_short_kernel<kDtype, kLayer, NV, kWaveRow>), grid, block, 0, s, a, columns, dw, db);
  }
};

// Whether dw and db are summed by columns rather than from parts (as measured above).
bool by_columns(int dtype, const Shape& sh, int64_t T, int64_t d) {
  if (!sh.wave && sh.nv * (dtype == 1 ? 8 : 4) > 8) return true;
  return T <= 1024 && T * d * (dtype == 1 ? 2 : 4) <= int64_t(10) << 20;
}
// Threads that a compute unit holds at up to 64 registers. Layer norms of one bf16
// vector to a thread have 66, of two 96, of four fp32 vectors 116: of these it holds
// fewer (from 7169 columns on one workgroup, not two), and what the grid has beyond
// them starts after the first ones have ended.
constexpr int64_t kResident = 2048;
constexpr int64_t kStreamBytes = int64_t(128) << 20;

}  // namespace

hipError_t launch_norm(int dtype, bool layer, const NormArgs& a, hipStream_t s) {
  const Shape sh = row_shape(dtype, a.d, 1024);
  const int64_t groups = sh.wave ? (a.T + 3) / 4 : a.T, most = 256 * (kResident / sh.threads);
  const dim3 grid(static_cast<unsigned>(groups < most ? groups : most));
  const int64_t bytes = a.T * a.d * (dtype == 1 ? 2 : 4) * (a.residual ? a.sum ? 4 : 3 : 2);
  by_type(dtype, layer, bytes >= kStreamBytes, sh, NormLaunch{a, grid, dim3(sh.threads), s});
  return hipGetLastError();
}

int norm_grad_parts(int dtype, int64_t T, int64_t d) {
  const Shape sh = row_shape(dtype, d, 1024);
  if (by_columns(dtype, sh, T, d)) return 0;
  // One workgroup to a compute unit, two of few threads: every part is written and
  // read once more. Measured with one, two, three: 4096 x 7168 42, 48, 52 us; 8192
  // x 4096 48, 51, 57; 16384 x 2048 66, 50, 53; 8192 x 512 12.6, 12.4, 14.0.
  const int64_t groups = sh.wave ? (T + 3) / 4 : T, most = sh.threads < 512 ? 512 : 256;
  return static_cast<int>(groups < most ? groups : most);
}

bool norm_grad_shifts(int dtype, bool layer, int64_t T, int64_t d) {
  const Shape sh = row_shape(dtype, d, 1024);
  return layer && !sh.wave && sh.nv * (dtype == 1 ? 8 : 4) > 8;
}

hipError_t launch_norm_grad(int dtype, bool layer, const NormGradArgs& a, float* dw, float* db, hipStream_t s) {
  const Shape sh = row_shape(dtype, a.d, 1024);
  const int parts = norm_grad_parts(dtype, a.T, a.d);
  const bool sums = dw || db;
  if (a.shift) {
    const int64_t groups = (a.T + 3) / 4;
    const dim3 grid(static_cast<unsigned>(groups < 2048 ? groups : 2048));
    if (dtype == 1) hipLaunchKernelGGL(norm_shift_kernel<1>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(norm_shift_kernel<0>, grid, dim3(256), 0, s, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (parts == 0) {
    const int columns = sums ? (a.d / (dtype == 1 ? 8 : 4) + 3) / 4 : 0;
    const int64_t groups = sh.wave ? (a.T + 3) / 4 : a.T;
    const int rows = static_cast<int>(groups < 1024 ? groups : 1024);
    // (where dx takes the place of what the columns read, they are summed first)
    const bool apart = sums && (a.dx == a.dy || a.dx == a.x);
    by_type(dtype, layer, false, sh,
            NormShortLaunch{a, columns, dw, db, dim3(columns + (apart ? 0 : rows)), dim3(sh.threads), s});
    if (apart) by_type(dtype, layer, false, sh, NormShortLaunch{a, 0, dw, db, dim3(rows), dim3(sh.threads), s});
    return hipGetLastError();
  }
  const dim3 grid(parts);
  const int64_t bytes = a.T * a.d * (dtype == 1 ? 2 : 4) * (a.dx_in ? 4 : 3);
  by_type(dtype, layer, bytes >= kStreamBytes, sh, NormGradLaunch{a, grid, dim3(sh.threads), s});
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (!dw && !db) return hipSuccess;
  hipLaunchKernelGGL(norm_parts_kernel, dim3((a.d + 15) / 16, db ? 2 : 1), dim3(parts > 256 ? 1024 : 256), 0, s,
                     a.part_w, a.part_b, parts, a.d, dw, db);
  return hipGetLastError();
}

}  // namespace moe
