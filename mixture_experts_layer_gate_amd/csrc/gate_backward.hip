// Gradients of the gate projection l = x Wg^T + bias for a dense logit gradient
// dl [T][E] (the balance losses reach every expert, so it has no zeros to skip):
//   dx[t]   = dx_in[t] + sum_e dl[t][e] Wg[e]
//   dWg[e]  = sum_t dl[t][e] x[t],   dbias[e] = sum_t dl[t][e]
//
// dl is fp32 and the matrix cores take bf16, so dl is written once as three bf16
// planes whose sum it is exactly (8 significant bits each: hi, then what hi
// leaves, then what both leave; the last rounds only denormals). dWg is an fp32
// result and takes all three planes: its products are then exact and its sums
// fp32. dx is a bf16 result and takes the first two: what it drops is below
// 2^-16 of each term, where its final rounding is up to 2^-8 of the sum.
//
// dWg sums over tokens, and both its operands are stored with the token as the
// slow index; the fragments' eight consecutive tokens per lane come from
// transposing LDS reads (ds_read_b64_tr_b16), as Wg's do in dx.
#include "common.h"
#include "router.h"

namespace moe {

namespace {

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kStep = 32;   // K per step (one MFMA)
constexpr int kCols = 128;  // output columns per workgroup
constexpr int kRowsX = 128; // tokens per dx workgroup

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
// experts per dWg workgroup
int dwg_rows(int E) { return E <= 64 ? 32 : 128; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  const uint32_t n = bytes <= 0 ? 0u : (bytes > 0xfffffff0ll ? 0xfffffff0u : static_cast<uint32_t>(bytes));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), static_cast<int>(n),
                                           0x00020000);
}
// 64 lanes x 16 bytes into LDS at dst (wave-uniform), lane order; zeros past the descriptor's end
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(dst), 16, off, 0, 0, 0);
}

// Slot of 16-byte chunk c of row k, for transposing reads (rows of 256 or 64
// bytes): each half-wave of a read then touches all 64 banks once.
template <int CPR>
__device__ __forceinline__ int tr_swz(int k) {
  return CPR == 16 ? (k % 4) * 4 + (k / 4) % 4 : ((k / 8) & 1) * 2;
}
// Fragment of 16 columns (from column col0) x 32 rows of a [32][CPR * 8] bf16
// tile: lane l gets column col0 + l % 16, rows 8 (l / 16) .. + 7.
template <int CPR>
__device__ __forceinline__ bf16x8_t frag_tr(const char* tile, int col0) {
  const int lane = threadIdx.x & 63;
  const int c = col0 / 8 + (lane % 4) / 2;
  i16x4_t half[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = 8 * (lane / 16) + 4 * h + (lane % 16) / 4;
    const char* p = tile + k * (CPR * 16) + (c ^ tr_swz<CPR>(k)) * 16 + (lane % 2) * 8;
    half[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(p));
  }
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// dl -> planes [3][Tp][Ep] (zero past T and E) and column sums of 16-row blocks.
constexpr int kSplitRows = 16;
__global__ __launch_bounds__(256) void split_kernel(const float* __restrict__ dl, int64_t T, int E, int64_t Tp, int Ep,
                                                    bf16_t* __restrict__ planes, float* __restrict__ bpart) {
  const int64_t plane = Tp * Ep;
  for (int64_t blk = blockIdx.x; blk < Tp / kSplitRows; blk += gridDim.x)
    for (int e = threadIdx.x; e < Ep; e += 256) {
      float v[kSplitRows], sum = 0.0f;
#pragma unroll
      for (int r = 0; r < kSplitRows; ++r) {
        const int64_t t = blk * kSplitRows + r;
        v[r] = t < T && e < E ? dl[t * E + e] : 0.0f;
      }
#pragma unroll
      for (int r = 0; r < kSplitRows; ++r) {
        const int64_t at = (blk * kSplitRows + r) * Ep + e;
        // hi by truncation: never past the largest finite value, exact remainder
        const uint32_t hb = __float_as_uint(v[r]) & 0xffff0000u;
        const bool fin = (hb & 0x7f800000u) != 0x7f800000u;
        const float r1 = fin ? v[r] - __uint_as_float(hb) : 0.0f;
        const uint32_t mb = __float_as_uint(r1) & 0xffff0000u;
        const float r2 = r1 - __uint_as_float(mb);
        // a NaN keeps a set mantissa bit
        const uint32_t h16 = (hb >> 16) | (v[r] != v[r] ? 0x40u : 0u);
        planes[at] = static_cast<bf16_t>(h16);
        planes[plane + at] = static_cast<bf16_t>(mb >> 16);
        planes[2 * plane + at] = static_cast<bf16_t>(f32_to_bf16_bits(r2));
        sum += v[r];
      }
      if (e < E) bpart[blk * E + e] = sum;
    }
}

// One BM-expert x 128-column tile of part blockIdx.z of the tokens.
template <int BM>
__global__ __launch_bounds__(256) void dwg_kernel(const bf16_t* __restrict__ x, const bf16_t* __restrict__ planes,
                                                  int64_t T, int64_t d, int E, int64_t Tp, int Ep, int64_t steps,
                                                  float* __restrict__ out) {
  constexpr int ACPR = BM / 8;                // 16-byte chunks per plane row
  constexpr int kA = 3 * kStep * BM * 2, kB = kStep * kCols * 2, kStage = kA + kB;
  constexpr int AI = kA / 1024, LI = kStage / 1024;  // load instructions of a stage: the planes', all
  constexpr int WM = BM == 128 ? 2 : 1, WN = 4 / WM;
  constexpr int MI = BM / WM / 16, NJ = kCols / WN / 16;
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int wm = wv / WN, wn = wv % WN;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kCols;
  const int e0 = blockIdx.y * BM;
  const int64_t s0 = steps * blockIdx.z / gridDim.z, s1 = steps * (blockIdx.z + 1) / gridDim.z;

  auto issue = [&](int64_t st, char* dst) {
    const int64_t t = st * kStep;
    const __amdgpu_buffer_rsrc_t rx = rsrc(x + t * d + n0, ((T - t) * d - n0) * 2);
#pragma unroll
    for (int q0 = 0; q0 < LI; q0 += 4) {
      const int q = q0 + wv;  // wave-uniform
      if (q < AI) {
        constexpr int RPI = 64 / ACPR;  // plane rows per instruction
        const int r = (q * RPI) % kStep + lane / ACPR;
        const int c = (lane % ACPR) ^ tr_swz<ACPR>(r);
        const bf16_t* base = planes + (static_cast<int64_t>((q * RPI) / kStep) * Tp + t) * Ep + e0;
        load_lds16(rsrc(base, (static_cast<int64_t>(kStep) * Ep) * 2), dst + q * 1024,
                   static_cast<uint32_t>((r * Ep + c * 8) * 2));
      } else if (q < LI) {
        const int r = (q - AI) * 4 + lane / 16, c = (lane % 16) ^ tr_swz<16>(r);
        load_lds16(rx, dst + q * 1024, static_cast<uint32_t>(r * d * 2 + c * 16));
      }
    }
  };

  f32x4_t acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  if (s0 < s1) issue(s0, lds);
  for (int64_t st = s0; st < s1; ++st) {
    char* cur = lds + ((st - s0) & 1) * kStage;
    char* nxt = lds + ((st - s0 + 1) & 1) * kStage;
    __syncthreads();  // stage st has landed for every wave, and every wave has read stage st - 1 out
    if (st + 1 < s1) issue(st + 1, nxt);
    bf16x8_t b[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) b[j] = frag_tr<16>(cur + kA, wn * (NJ * 16) + j * 16);
#pragma unroll
    for (int pl = 2; pl >= 0; --pl)
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const bf16x8_t a = frag_tr<ACPR>(cur + pl * (kStep * BM * 2), wm * (MI * 16) + i * 16);
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[j], acc[i][j], 0, 0, 0);
      }
  }
  float* o = out + static_cast<int64_t>(blockIdx.z) * E * d;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int e = e0 + wm * (MI * 16) + i * 16 + 4 * (lane / 16) + v;
      if (e >= E) continue;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t n = n0 + wn * (NJ * 16) + j * 16 + lane % 16;
        if (n < d) o[e * d + n] = acc[i][j][v];
      }
    }
}

// Parts summed in order (parts > 0), and dbias from the 16-row blocks' sums.
__global__ __launch_bounds__(256) void dwg_sum_kernel(const float* __restrict__ part, int parts, int64_t n4,
                                                      float* __restrict__ dwg, const float* __restrict__ bpart,
                                                      int64_t blocks, int E, float* __restrict__ dbias,
                                                      int bias_groups) {
  if (static_cast<int>(blockIdx.x) < bias_groups) {
    // 16 experts per workgroup: 16 slices of blocks, then the slices in order
    __shared__ double sp[16][16];
    const int el = threadIdx.x % 16, sl = threadIdx.x / 16;
    const int e = blockIdx.x * 16 + el;
    double v = 0.0;
    if (e < E)
      for (int64_t r = sl; r < blocks; r += 16) v += bpart[r * E + e];
    sp[sl][el] = v;
    __syncthreads();
    if (threadIdx.x < 16 && e < E) {
      double t = 0.0;
      for (int q = 0; q < 16; ++q) t += sp[q][threadIdx.x];
      dbias[e] = static_cast<float>(t);
    }
    return;
  }
  if (parts < 2) return;
  const int64_t stride = static_cast<int64_t>(gridDim.x - bias_groups) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x - bias_groups) * 256 + threadIdx.x; i < n4; i += stride) {
    f32x4_t v = reinterpret_cast<const f32x4_t*>(part)[i];
    for (int p = 1; p < parts; ++p) v += reinterpret_cast<const f32x4_t*>(part)[p * n4 + i];
    reinterpret_cast<f32x4_t*>(dwg)[i] = v;
  }
}

// One 128-token x 128-column tile of dx: K = the experts, planes hi and mid.
__global__ __launch_bounds__(256) void gate_dx_kernel(const bf16_t* __restrict__ planes, const bf16_t* __restrict__ wg,
                                                      const bf16_t* dx_in, int64_t T, int64_t d, int E, int64_t Tp,
                                                      int Ep, bf16_t* dx) {
  constexpr int kA = 2 * kRowsX * kStep * 2, kB = kStep * kCols * 2, kStage = kA + kB;
  constexpr int AI = kA / 1024, LI = kStage / 1024;
  constexpr int MI = 4, NJ = 4;
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int wm = wv / 2, wn = wv % 2;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kCols;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kRowsX;
  const int steps = (E + kStep - 1) / kStep;

  auto issue = [&](int st, char* dst) {
    const int k0 = st * kStep;
    const __amdgpu_buffer_rsrc_t rw =
        rsrc(wg + static_cast<int64_t>(k0) * d + n0, (static_cast<int64_t>(E - k0) * d - n0) * 2);
#pragma unroll
    for (int q0 = 0; q0 < LI; q0 += 4) {
      const int q = q0 + wv;
      if (q < AI) {
        // 16 rows of 64 bytes; chunk c of row r in slot c ^ (r / 4) % 4
        const int pl = q / (AI / 2), r = (q % (AI / 2)) * 16 + lane / 4, c = (lane % 4) ^ ((r / 4) % 4);
        const bf16_t* base = planes + (static_cast<int64_t>(pl) * Tp + t0) * Ep + k0;
        load_lds16(rsrc(base, (static_cast<int64_t>(kRowsX) * Ep) * 2), dst + q * 1024,
                   static_cast<uint32_t>((r * Ep + c * 8) * 2));
      } else {
        const int r = (q - AI) * 4 + lane / 16, c = (lane % 16) ^ tr_swz<16>(r);
        load_lds16(rw, dst + q * 1024, static_cast<uint32_t>(r * d * 2 + c * 16));
      }
    }
  };

  f32x4_t acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  issue(0, lds);
  for (int st = 0; st < steps; ++st) {
    char* cur = lds + (st & 1) * kStage;
    char* nxt = lds + ((st + 1) & 1) * kStage;
    __syncthreads();
    if (st + 1 < steps) issue(st + 1, nxt);
    bf16x8_t b[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) b[j] = frag_tr<16>(cur + kA, wn * 64 + j * 16);
#pragma unroll
    for (int pl = 1; pl >= 0; --pl)
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int r = wm * 64 + i * 16 + lane % 16, c = (lane / 16) ^ ((r / 4) % 4);
        const bf16x8_t a =
            *reinterpret_cast<const bf16x8_t*>(cur + pl * (kRowsX * kStep * 2) + r * (kStep * 2) + c * 16);
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[j], acc[i][j], 0, 0, 0);
      }
  }
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t t = t0 + wm * 64 + i * 16 + 4 * (lane / 16) + v;
      if (t >= T) continue;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t n = n0 + wn * 64 + j * 16 + lane % 16;
        if (n >= d) continue;
        float r = acc[i][j][v];
        if (dx_in) r += __uint_as_float(static_cast<uint32_t>(dx_in[t * d + n]) << 16);
        reinterpret_cast<__bf16*>(dx)[t * d + n] = static_cast<__bf16>(r);
      }
    }
}

struct GateWs {
  int64_t Tp, blocks, steps;
  int Ep, bm, parts;
  bf16_t* planes;
  float* bpart;
  float* part;  // null when one part: the sums go straight to dwg
};

size_t layout(int64_t T, int64_t d, int E, void* ws, GateWs* g) {
  auto at = [&](size_t off) { return ws ? static_cast<char*>(ws) + off : nullptr; };
  auto pad = [](size_t v) { return (v + 255) / 256 * 256; };
  g->bm = dwg_rows(E);
  g->Ep = static_cast<int>(up(E, g->bm));
  g->Tp = up(T, kRowsX);
  g->blocks = g->Tp / kSplitRows;
  g->steps = (T + kStep - 1) / kStep;
  // token parts: about one round of workgroups, at least 8 steps to each
  const int64_t tiles = (d + kCols - 1) / kCols * (g->Ep / g->bm);
  int64_t parts = (256 + tiles - 1) / tiles;
  if (parts > g->steps / 8) parts = g->steps / 8;
  g->parts = parts < 1 ? 1 : static_cast<int>(parts);
  size_t off = 0;
  g->planes = reinterpret_cast<bf16_t*>(at(off));
  off += pad(size_t(3) * g->Tp * g->Ep * 2);
  g->bpart = reinterpret_cast<float*>(at(off));
  off += pad(size_t(g->blocks) * E * 4);
  g->part = g->parts > 1 ? reinterpret_cast<float*>(at(off)) : nullptr;
  if (g->parts > 1) off += pad(size_t(g->parts) * E * d * 4);
  return off;
}

}  // namespace

size_t gate_backward_ws(int64_t T, int64_t d, int E) {
  GateWs g{};
  return layout(T, d, E, nullptr, &g);
}

hipError_t launch_gate_backward(const void* x, const void* wg, const float* dlogits, const void* dx_in, void* dx,
                                float* dwg, float* dbias, int64_t T, int64_t d, int E, void* ws, hipStream_t s) {
  GateWs g{};
  layout(T, d, E, ws, &g);
  const bf16_t* xb = static_cast<const bf16_t*>(x);
  const unsigned ncols = static_cast<unsigned>((d + kCols - 1) / kCols);
  hipLaunchKernelGGL(split_kernel, dim3(static_cast<unsigned>(g.blocks < (1 << 20) ? g.blocks : (1 << 20))), dim3(256),
                     0, s, dlogits, T, E, g.Tp, g.Ep, g.planes, g.bpart);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  float* o = g.parts > 1 ? g.part : dwg;
  const dim3 grid(ncols, g.Ep / g.bm, g.parts);
  if (g.bm == 32)
    hipLaunchKernelGGL(dwg_kernel<32>, grid, dim3(256), 0, s, xb, g.planes, T, d, E, g.Tp, g.Ep, g.steps, o);
  else
    hipLaunchKernelGGL(dwg_kernel<128>, grid, dim3(256), 0, s, xb, g.planes, T, d, E, g.Tp, g.Ep, g.steps, o);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  const int bias_groups = (E + 15) / 16;
  const int64_t n4 = static_cast<int64_t>(E) * d / 4;
  const int64_t sum_groups = g.parts > 1 ? ((n4 + 255) / 256 < 2048 ? (n4 + 255) / 256 : 2048) : 0;
  hipLaunchKernelGGL(dwg_sum_kernel, dim3(static_cast<unsigned>(bias_groups + sum_groups)), dim3(256), 0, s, g.part,
                     g.parts, n4, dwg, g.bpart, g.blocks, E, dbias, bias_groups);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  hipLaunchKernelGGL(gate_dx_kernel, dim3(ncols, static_cast<unsigned>(g.Tp / kRowsX)), dim3(256), 0, s, g.planes,
                     static_cast<const bf16_t*>(wg), static_cast<const bf16_t*>(dx_in), T, d, E, g.Tp, g.Ep,
                     static_cast<bf16_t*>(dx));
  return hipGetLastError();
}

}  // namespace moe
