// Device-side helpers shared by the kernels of the MoE-layer library (gfx950, wave64).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

typedef uint16_t bf16_t;  // bf16 storage: the upper 16 bits of an fp32

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) unsigned int u32x4_t;

constexpr int kWave = 64;

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// fp32 -> bf16, round to nearest even (finite inputs)
__device__ __forceinline__ uint32_t f32_to_bf16_bits(float f) {
  uint32_t u = __float_as_uint(f);
  u += 0x7fffu + ((u >> 16) & 1u);
  return u >> 16;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  return f32_to_bf16_bits(lo) | (f32_to_bf16_bits(hi) << 16);
}

// Element traits: storage type and its conversion to/from fp32.
template <int kDtype> struct Elt;
template <> struct Elt<0> {  // fp32
  typedef float T;
  static constexpr int kBytes = 4;
};
template <> struct Elt<1> {  // bf16
  typedef bf16_t T;
  static constexpr int kBytes = 2;
};

// ---------------- LDS-staged matrix products ----------------
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                           static_cast<int>(bytes), 0x00020000);
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// Every LDS read of this wave has returned (lgkmcnt 0; vmcnt and expcnt left alone).
__device__ __forceinline__ void wait_lds_reads() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// Workgroup barrier without the memory fence __syncthreads() carries: that fence
// makes the compiler wait for every outstanding load, including the LDS stages
// still being prefetched. LDS readiness is handled by explicit vmcnt waits
// before the barrier; the empty asm keeps the compiler from moving memory
// operations across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Swizzle of the 16-byte chunks of row k of a [K][256] bf16 LDS stage: chunk c
// of row k sits in slot c ^ f(k). The transposing reads of a B fragment touch
// 16 rows k = 8g + 4h + i (g, i in 0..3) at the same columns; f spreads every
// half-wave over all 64 banks.
__device__ __forceinline__ int kn_swz(int k) { return (k % 4) * 4 + (k / 4) % 4; }

typedef short i16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float silu_mul(float g, float u) {
  // SiLU(g) * u = g / (1 + exp(-g)) * u
  return g / (1.0f + __expf(-g)) * u;
}

}  // namespace moe
