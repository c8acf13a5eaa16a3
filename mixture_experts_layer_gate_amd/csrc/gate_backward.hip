// Gradients of the gate projection l = x Wg^T + bias for a dense logit gradient
// dl [T][E] (the balance losses reach every expert, so it has no zeros to skip):
//   dx[t]   = dx_in[t] + sum_e dl[t][e] Wg[e]
//   dWg[e]  = sum_t dl[t][e] x[t],   dbias[e] = sum_t dl[t][e]
//
// dl is fp32 and the matrix cores take bf16, so dl is written once as three bf16
// planes whose sum it is exactly (8 significant bits each: hi, truncated, then
// what hi leaves, to nearest, then what both leave; the last rounds only
// denormals). dWg is an fp32 result and takes all three planes: its products are
// then exact and its sums fp32. dx is a bf16 result and takes the first two: what
// it drops is at most 2^-16 of each term (mid's last bit is 2^-15 of dl's first,
// at most), where its final rounding is up to 2^-8 of the sum: it shows where the
// terms cancel by more than some 2^8. The third plane was measured: 4096 x 7168 x 256
// 84 -> 96 us, 32 x 7168 x 256 11.7 -> 13.1, 2047 x 6144 x 16 21.7 -> 22.1.
//
// An infinity in x or Wg meets planes that are zero or of the other sign, which
// would make a NaN of the formula's infinity (and so may products past fp32's
// range). Each non-finite result is therefore formed again from dl itself, term by
// term: no finite result can come of such products, so nothing else is looked at.
// (Asking every accumulator costs 0.2 to 0.9 us a call: 2047 x 6144 x 16 21.6 -> 21.8,
// 8192 x 4096 x 64 47.0 -> 47.9, 32 x 7168 x 256 11.2 -> 11.7, 4096 x 7168 x 256 the
// same. With one infinite row of x the last takes 1.4 ms, with nothing else in x and Wg 1.9.)
//
// dWg sums over tokens, and both its operands come with the token as the slow
// index: the planes are written transposed as well, and x's fragments (eight
// consecutive tokens per lane) come from transposing LDS reads
// (ds_read_b64_tr_b16), as Wg's do in dx. Those reads are written as assembly
// that waits for its own results: for the builtin the compiler waits until no
// load into LDS is in flight, which takes the loads' lead away.
//
// Measured at 4096 x 7168 x 256: dWg 46 us (45 GFLOP in bf16, 980 TFLOP/s; its
// matrix products alone take 20 us of matrix-core time, the loads alone about 26
// us, and they overlap in part), dx with dWg's parts 38 us (118 MB, 3.1 TB/s; 30
// GFLOP), the split 6 us.
#include "common.h"
#include "router.h"

namespace moe {

namespace {

constexpr int kStep = 32;    // K of one step (one MFMA)
constexpr int kRowsX = 128;  // tokens per dx workgroup
constexpr int kColsX = 128;  // columns per dx workgroup

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  return make_rsrc(base, bytes <= 0 ? 0u : (bytes > 0xfffffff0ll ? 0xfffffff0u : static_cast<uint32_t>(bytes)));
}
// 64 lanes x 16 bytes into LDS at dst (wave-uniform), lane order; zeros past the descriptor's end
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(dst), 16, off, 0, 0, 0);
}

// Four fragments of 16 columns (col0, col0 + 16, ..) x 32 rows of a [32][CPR * 8]
// bf16 tile whose 16-byte chunk c of row k sits in slot c ^ kn_swz(k): lane l
// gets column l % 16, rows 8 (l / 16) .. + 7 of each. `at` holds the lane's byte
// offsets inside the tile (fixed through the K loop).
template <int CPR>
__device__ __forceinline__ void tr_offsets(int col0, uint32_t (&at)[8]) {
  static_assert(CPR == 16 || CPR == 32, "rows of 256 or 512 bytes");
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = (col0 + i * 16) / 8 + (lane % 4) / 2;
      const int k = 8 * (lane / 16) + 4 * h + (lane % 16) / 4;
      at[2 * i + h] = static_cast<uint32_t>(k * (CPR * 16) + ((c ^ kn_swz(k)) % CPR) * 16 + (lane % 2) * 8);
    }
}
__device__ __forceinline__ void tr_read(const char* tile, const uint32_t (&at)[8], bf16x8_t (&frag)[4]) {
  const uint32_t base =
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(tile)));
  i16x4_t r[8];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8\n\t"
      "ds_read_b64_tr_b16 %1, %9\n\t"
      "ds_read_b64_tr_b16 %2, %10\n\t"
      "ds_read_b64_tr_b16 %3, %11\n\t"
      "ds_read_b64_tr_b16 %4, %12\n\t"
      "ds_read_b64_tr_b16 %5, %13\n\t"
      "ds_read_b64_tr_b16 %6, %14\n\t"
      "ds_read_b64_tr_b16 %7, %15\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
      : "v"(base + at[0]), "v"(base + at[1]), "v"(base + at[2]), "v"(base + at[3]), "v"(base + at[4]),
        "v"(base + at[5]), "v"(base + at[6]), "v"(base + at[7])
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i)
    frag[i] = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(r[2 * i], r[2 * i + 1], 0, 1, 2, 3, 4, 5, 6, 7));
}
// Stage rows of 32 K values, four 16-byte chunks: chunk c of row r in slot
// c ^ row_swz(r), so that a fragment's reads (lane l: row l % 16, chunk l / 16)
// touch all banks evenly, both for 16 consecutive lanes and for the lanes the
// hardware takes together in a 16-byte read (0-3, 12-15, 20-27; 4-11, 16-19,
// 28-31; the same above 32): no conflicts counted, where c ^ (r / 4) % 4 doubled
// the reads' time.
__device__ __forceinline__ int row_swz(int r) {
  const int q = (r / 4) % 4;  // 0, 2, 3, 1 for q = 0 .. 3
  return (q >> 1) | (((q ^ (q >> 1)) & 1) << 1);
}
__device__ __forceinline__ bf16x8_t row_frag(const char* tile, int row0) {
  const int lane = threadIdx.x & 63, r = row0 + lane % 16;
  return *reinterpret_cast<const bf16x8_t*>(tile + r * (kStep * 2) + ((lane / 16) ^ row_swz(r)) * 16);
}

// One step's products: acc[i][j] += (transposed fragment i) x (row fragment j),
// summed over the planes, the smallest first; a plane's fragments are read while
// the one before it multiplies.
template <int kPlanes>
__device__ __forceinline__ void step_products(const char* rows, int plane_bytes, int row0, const char* cols,
                                              const uint32_t (&at)[8], f32x4_t (&acc)[4][4]) {
  bf16x8_t b[4], a[2][4];
  tr_read(cols, at, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) a[0][j] = row_frag(rows + (kPlanes - 1) * plane_bytes, row0 + j * 16);
#pragma unroll
  for (int p = 0; p < kPlanes; ++p) {
    if (p + 1 < kPlanes) {
#pragma unroll
      for (int j = 0; j < 4; ++j) a[(p + 1) & 1][j] = row_frag(rows + (kPlanes - 2 - p) * plane_bytes, row0 + j * 16);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[i], a[p & 1][j], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Tile of workgroup `id` of n: consecutive tiles on one XCD (workgroup id runs
// on XCD id mod 8), so that tiles sharing an operand share an L2.
__device__ __forceinline__ int xcd_tile(int id, int n) {
  const int per = n / 8;
  return id < 8 * per ? (id % 8) * per + id / 8 : id;
}

// One pipelined K loop: `issue(buffer)` starts the next step's loads (PER of them
// per wave) into one of NST stage buffers, `work(buffer)` multiplies it. The
// loads run NST - 1 steps ahead; a step's own are the oldest in flight.
template <int NST, int PER, int kStage, typename Issue, typename Work>
__device__ __forceinline__ void pipeline(int steps, char* lds, Issue&& issue, Work&& work) {
#pragma unroll
  for (int p = 0; p < NST - 1; ++p)
    if (p < steps) issue(lds + p * kStage);
  int buf = 0, ahead = NST - 1;
  for (int st = 0; st < steps; ++st) {
    if (st + NST - 2 < steps)
      wait_vmcnt<(NST - 2) * PER>();
    else
      wait_vmcnt<0>();
    wait_lds_reads();  // of the step before: its buffer is refilled below
    lds_barrier();
    if (st + NST - 1 < steps) issue(lds + ahead * kStage);
    work(lds + buf * kStage);
    buf = buf + 1 == NST ? 0 : buf + 1;
    ahead = ahead + 1 == NST ? 0 : ahead + 1;
  }
}

// One 64-token x 64-expert block: dl -> rows [Ep / 32][2][Tp][32] (hi, mid by
// blocks of 32 experts: dx's operand) and cols [Tp / 32][3][Ep][32] (all planes
// by blocks of 32 tokens, transposed through LDS: dWg's), zero past T and E, and
// the block's column sums. A step's operand is thus one contiguous piece per
// plane; in plain rows a tile's 128 rows lie a power of two apart and meet in
// few of the L2's channels.
constexpr int kBlk = 64;
__global__ __launch_bounds__(256) void split_kernel(const float* __restrict__ dl, int64_t T, int E, int64_t Tp, int Ep,
                                                    bf16_t* __restrict__ rows, bf16_t* __restrict__ cols,
                                                    float* __restrict__ bpart) {
  constexpr int kPitch = kBlk + 8;
  __shared__ __attribute__((aligned(16))) bf16_t tr[3][kBlk * kPitch];
  __shared__ float part[16][kBlk];
  const int64_t tb = static_cast<int64_t>(blockIdx.y) * kBlk;
  const int eb = blockIdx.x * kBlk;
  const int cg = (threadIdx.x % 16) * 4, rg = (threadIdx.x / 16) * 4;  // 4 rows x 4 columns of the block
  const bool vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(dl) & 15) == 0;
  const int e = eb + cg;
  float v[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t t = tb + rg + r;
    if (vec) {
      const f32x4_t u = t < T && e < E ? *reinterpret_cast<const f32x4_t*>(dl + t * E + e) : f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) v[r][c] = u[c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[r][c] = t < T && e + c < E ? dl[t * E + e + c] : 0.0f;
    }
  }
  uint32_t p[3][4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // hi by truncation: never past the largest finite value, exact remainder
      const uint32_t hb = __float_as_uint(v[r][c]) & 0xffff0000u;
      const bool fin = (hb & 0x7f800000u) != 0x7f800000u;
      const float r1 = fin ? v[r][c] - __uint_as_float(hb) : 0.0f;
      // mid to nearest: what dx drops is then at most 2^-16 of dl
      const uint32_t mb = static_cast<uint32_t>(f32_to_bf16_bits(r1)) << 16;
      p[0][r][c] = (hb >> 16) | (v[r][c] != v[r][c] ? 0x40u : 0u);  // a NaN keeps a set mantissa bit
      p[1][r][c] = mb >> 16;
      p[2][r][c] = f32_to_bf16_bits(r1 - __uint_as_float(mb));
    }
#pragma unroll
  for (int pl = 0; pl < 2; ++pl)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<uint2*>(rows + ((e / kStep * 2 + pl) * Tp + tb + rg + r) * kStep + e % kStep) =
          make_uint2(p[pl][r][0] | (p[pl][r][1] << 16), p[pl][r][2] | (p[pl][r][3] << 16));
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int pl = 0; pl < 3; ++pl)
      *reinterpret_cast<uint2*>(&tr[pl][(cg + c) * kPitch + rg]) =
          make_uint2(p[pl][0][c] | (p[pl][1][c] << 16), p[pl][2][c] | (p[pl][3][c] << 16));
    part[threadIdx.x / 16][cg + c] = ((v[0][c] + v[1][c]) + v[2][c]) + v[3][c];
  }
  __syncthreads();
#pragma unroll
  for (int pl = 0; pl < 3; ++pl)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = q * 32 + threadIdx.x / 8, c = (threadIdx.x % 8) * 8;
      *reinterpret_cast<u32x4_t*>(cols + (((tb + c) / kStep * 3 + pl) * Ep + eb + r) * kStep + c % kStep) =
          *reinterpret_cast<const u32x4_t*>(&tr[pl][r * kPitch + c]);
    }
  if (threadIdx.x < kBlk && eb + static_cast<int>(threadIdx.x) < E) {
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < 16; ++q) sum += part[q][threadIdx.x];
    bpart[static_cast<int64_t>(blockIdx.y) * E + eb + threadIdx.x] = sum;
  }
}

struct GateArgs {
  const bf16_t* x;
  const bf16_t* wg;
  const bf16_t* dx_in;
  bf16_t* dx;
  const float* dl;
  const bf16_t* rows;  // split_kernel's outputs
  const bf16_t* cols;
  float* out;  // dwg, or its parts [parts][E][d]
  int64_t T, d, Tp;
  int E, Ep;
  int steps, etiles, parts, w_tiles;  // dWg: 32-token steps, expert tiles, token parts, tiles in all
  int ncols, x_tiles;                 // dx: column tiles, tiles in all
};

__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= 3.402823466e38f; }

// A BM-expert x BN-column tile of one part of the tokens: out[part][e][n].
// BM / 64 x BN / 64 waves, each 64 experts x 64 columns.
template <int BM, int BN, int NST>
struct DwgTile {
  static constexpr int kPlane = kStep * BM * 2, kA = 3 * kPlane, kB = kStep * BN * 2, kStage = kA + kB;
  static constexpr int kLds = NST * kStage;
  __device__ static __forceinline__ void run(const GateArgs& g, int id, char* lds);
};
template <int BM, int BN, int NST>
__device__ __forceinline__ void DwgTile<BM, BN, NST>::run(const GateArgs& g, int id, char* lds) {
  const int64_t T = g.T, d = g.d;
  const int E = g.E, Ep = g.Ep, steps = g.steps, etiles = g.etiles, parts = g.parts;
  constexpr int WN = BN / 64, NW = BM / 64 * WN;
  constexpr int BCPR = BN / 8;  // 16-byte chunks of a stage row of x
  constexpr int AI = kA / 1024 / NW, BI = kB / 1024 / NW, PER = AI + BI;  // load instructions of a wave
  static_assert(AI * NW * 1024 == kA && BI * NW * 1024 == kB, "every wave loads as much");
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / WN, wn = wv % WN;
  // expert tiles of one column block next to each other (they read the same x),
  // parts outermost (an XCD's tiles then read one or two parts of the planes,
  // which its L2 holds)
  const int tile = xcd_tile(id, g.w_tiles);
  const int e0 = tile % etiles * BM;
  const int ncols = static_cast<int>((d + BN - 1) / BN);
  const int64_t n0 = static_cast<int64_t>(tile / etiles % ncols) * BN;
  const int part = tile / etiles / ncols;
  // the first steps % parts parts take one step more
  const int s0 = part * (steps / parts) + min(part, steps % parts);
  const int n_steps = steps / parts + (part < steps % parts);

  // Operand bases of the next step to load, advanced as steps are issued (in
  // order): one 64-bit addition each in front of a step's loads.
  const int64_t t0 = static_cast<int64_t>(s0) * kStep;
  const bf16_t* xb = g.x + t0 * d + n0;
  int64_t x_bytes = ((T - t0) * d - n0) * 2;  // to x's end: rows past T read as zeros
  const bf16_t* cb = g.cols + (static_cast<int64_t>(s0) * 3 * Ep + e0) * kStep;
  uint32_t aoff[AI], boff[BI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    constexpr int IPP = BM / 16;  // instructions per plane, 16 rows of 64 bytes each
    const int r = ((wv * AI + i) % IPP) * 16 + lane / 4;
    aoff[i] = static_cast<uint32_t>((r * 4 + ((lane % 4) ^ row_swz(r))) * 16);
  }
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    constexpr int RPI = 64 / BCPR;
    const int r = (wv * BI + i) * RPI + lane / BCPR;
    boff[i] = static_cast<uint32_t>(r * d * 2 + (((lane % BCPR) ^ kn_swz(r)) % BCPR) * 16);
  }
  auto issue = [&](char* dst) {
    const __amdgpu_buffer_rsrc_t rx = rsrc(xb, x_bytes);
#pragma unroll
    for (int i = 0; i < AI; ++i) {
      const int q = wv * AI + i, pl = q / (BM / 16);
      load_lds16(rsrc(cb + pl * Ep * kStep, BM * kStep * 2), dst + q * 1024, aoff[i]);
    }
#pragma unroll
    for (int i = 0; i < BI; ++i) load_lds16(rx, dst + kA + (wv * BI + i) * 1024, boff[i]);
    xb += kStep * d;
    x_bytes -= kStep * d * 2;
    cb += 3 * Ep * kStep;
  };
  f32x4_t acc[4][4];  // [column block][expert block]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  uint32_t at[8];
  tr_offsets<BCPR>(wn * 64, at);
  pipeline<NST, PER, kStage>(n_steps, lds, issue, [&](const char* cur) {
    step_products<3>(cur, kPlane, wm * 64, cur + kA, at, acc);
  });
  // accumulator of lane l: columns 4 (l / 16) .. + 3 of expert l % 16
  float* o = g.out + static_cast<int64_t>(part) * E * d;
  f32x4_t odd = {0.0f, 0.0f, 0.0f, 0.0f};  // NaN once an accumulator is not finite (four chains)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = e0 + wm * 64 + j * 16 + lane % 16;
    if (e >= E) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t n = n0 + wn * 64 + i * 16 + 4 * (lane / 16);
      if (n >= d) continue;
      *reinterpret_cast<f32x4_t*>(o + e * d + n) = acc[i][j];
#pragma unroll
      for (int q = 0; q < 4; ++q) odd[q] = __builtin_fmaf(acc[i][j][q], 0.0f, odd[q]);
    }
  }
  if (!__ballot((odd[0] + odd[1]) + (odd[2] + odd[3]) != 0.0f)) return;
  // each of them again, in token order (a lane reads what it has just written)
  const int64_t t1 = min(T, t0 + static_cast<int64_t>(n_steps) * kStep);
  for (int b = 0; b < 16; ++b) {
    const int e = e0 + wm * 64 + b / 4 * 16 + lane % 16;
    const int64_t n = n0 + wn * 64 + b % 4 * 16 + 4 * (lane / 16);
    if (e >= E || n >= d) continue;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(o + e * d + n);
    if (finite(v[0]) && finite(v[1]) && finite(v[2]) && finite(v[3])) continue;
    f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8  // loads in flight together
    for (int64_t t = t0; t < t1; ++t) {
      const float a = g.dl[t * E + e];
      const uint2 u = *reinterpret_cast<const uint2*>(g.x + t * d + n);
      sum[0] = __builtin_fmaf(a, bf16_lo(u.x), sum[0]);
      sum[1] = __builtin_fmaf(a, bf16_hi(u.x), sum[1]);
      sum[2] = __builtin_fmaf(a, bf16_lo(u.y), sum[2]);
      sum[3] = __builtin_fmaf(a, bf16_hi(u.y), sum[3]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = finite(v[q]) ? v[q] : sum[q];
    *reinterpret_cast<f32x4_t*>(o + e * d + n) = v;
  }
}

// What else there is to do: dbias from the 64-token blocks' sums, and, behind dWg,
// its parts summed in order.
struct SumArgs {
  const float* part;
  int parts;  // 1: dwg is whole already
  int64_t n4;
  float* dwg;
  const float* bpart;
  int blocks;
  float* dbias;
  int bias_groups, groups;  // workgroups: for dbias, in all
};
__device__ __forceinline__ void sum_group(const SumArgs& a, int group, int E, char* lds) {
  if (group < a.bias_groups) {
    // 16 experts per workgroup: 16 slices of blocks, then the slices in order
    double* sp = reinterpret_cast<double*>(lds);
    const int el = threadIdx.x % 16, sl = threadIdx.x / 16;
    const int e = group * 16 + el;
    double v = 0.0;
    if (e < E)
      for (int r = sl; r < a.blocks; r += 16) v += a.bpart[static_cast<int64_t>(r) * E + e];
    sp[sl * 16 + el] = v;
    __syncthreads();
    if (threadIdx.x < 16 && e < E) {
      double t = 0.0;
      for (int q = 0; q < 16; ++q) t += sp[q * 16 + threadIdx.x];
      a.dbias[e] = static_cast<float>(t);
    }
    return;
  }
  const int64_t stride = static_cast<int64_t>(a.groups - a.bias_groups) * 256;
  for (int64_t i = static_cast<int64_t>(group - a.bias_groups) * 256 + threadIdx.x; i < a.n4; i += stride) {
    f32x4_t v = reinterpret_cast<const f32x4_t*>(a.part)[i];
#pragma unroll 4  // loads in flight together (2047 x 6144 x 16, ten parts: the call 24.7 -> 23.2 us)
    for (int p = 1; p < a.parts; ++p) v += reinterpret_cast<const f32x4_t*>(a.part)[p * a.n4 + i];
    reinterpret_cast<f32x4_t*>(a.dwg)[i] = v;
  }
}

// One 128-token x 128-column tile of dx: K = the experts, planes hi and mid.
template <int NST>
struct DxTile {
  static constexpr int kPlane = kRowsX * kStep * 2, kA = 2 * kPlane, kB = kStep * kColsX * 2, kStage = kA + kB;
  static constexpr int kLds = NST * kStage;
  __device__ static __forceinline__ void run(const GateArgs& g, int tile, char* lds);
};
template <int NST>
__device__ __forceinline__ void DxTile<NST>::run(const GateArgs& g, int tile, char* lds) {
  constexpr int AI = kA / 1024 / 4, BI = kB / 1024 / 4, PER = AI + BI, BCPR = kColsX / 8;
  const int64_t T = g.T, d = g.d, Tp = g.Tp;
  const int E = g.E;
  const bf16_t* dx_in = g.dx_in;
  bf16_t* dx = g.dx;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / 2, wn = wv % 2;
  const int64_t n0 = static_cast<int64_t>(tile % g.ncols) * kColsX;
  const int64_t t0 = static_cast<int64_t>(tile / g.ncols) * kRowsX;

  // dx_in's rows as the epilogue takes them, those of the first two of its four
  // blocks read beside the first stage, the others two blocks ahead: read behind
  // the K loop they kept each tile waiting (the whole call 91.5 against 89.8 us at
  // 4096 x 7168 x 256, 53.4 against 51.4 at 8192 x 4096 x 64; all four ahead take
  // the registers of a third wave per SIMD).
  const int tr = lane / 8;
  const int64_t n = n0 + wn * 64 + (lane % 8) * 8;
  const bool col = n < d;
  u32x4_t in[2][2];
  auto read_in = [&](int j) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int64_t t = t0 + wm * 64 + j * 16 + p * 8 + tr;
      in[j % 2][p] = u32x4_t{0, 0, 0, 0};
      if (dx_in && col && t < T) in[j % 2][p] = *reinterpret_cast<const u32x4_t*>(dx_in + t * d + n);
    }
  };
  read_in(0);
  read_in(1);

  // operand bases of the next step to load, as for dWg
  const bf16_t* wb = g.wg + n0;
  int64_t w_bytes = (E * d - n0) * 2;  // rows past E read as zeros
  const bf16_t* rb = g.rows + t0 * kStep;
  uint32_t aoff[AI], boff[BI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int r = ((wv * AI + i) % (2 * AI)) * 16 + lane / 4;
    aoff[i] = static_cast<uint32_t>((r * 4 + ((lane % 4) ^ row_swz(r))) * 16);
  }
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    constexpr int RPI = 64 / BCPR;
    const int r = (wv * BI + i) * RPI + lane / BCPR;
    boff[i] = static_cast<uint32_t>(r * d * 2 + (((lane % BCPR) ^ kn_swz(r)) % BCPR) * 16);
  }
  auto issue = [&](char* dst) {
    const __amdgpu_buffer_rsrc_t rw = rsrc(wb, w_bytes);
#pragma unroll
    for (int i = 0; i < AI; ++i) {
      const int q = wv * AI + i, pl = q / (2 * AI);
      load_lds16(rsrc(rb + pl * Tp * kStep, kRowsX * kStep * 2), dst + q * 1024, aoff[i]);
    }
#pragma unroll
    for (int i = 0; i < BI; ++i) load_lds16(rw, dst + kA + (wv * BI + i) * 1024, boff[i]);
    wb += kStep * d;
    w_bytes -= kStep * d * 2;
    rb += 2 * Tp * kStep;
  };
  f32x4_t acc[4][4];  // [column block][token block]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  uint32_t at[8];
  tr_offsets<BCPR>(wn * 64, at);
  pipeline<NST, PER, kStage>((E + kStep - 1) / kStep, lds, issue, [&](const char* cur) {
    step_products<2>(cur, kPlane, wm * 64, cur + kA, at, acc);
  });
  // Accumulator of lane l: columns 4 (l / 16) .. + 3 of token l % 16. Through the
  // stage buffers (a wave's own 16 x 64 block at a time) to eight consecutive
  // columns per lane, so that loads and stores are whole 128-byte lines: with
  // the 8-byte accesses of the accumulator layout reading dx_in and writing dx
  // took 38 us at 4096 x 7168 x 32, this way 25.
  constexpr int kPitch = 64 + 4;
  __syncthreads();  // every wave has read the last stage
  float* ct = reinterpret_cast<float*>(lds) + wv * (16 * kPitch);
  uint32_t again = 0;  // rows of this lane left out, one bit to each
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x4_t own[2] = {in[j % 2][0], in[j % 2][1]};
    if (j < 2) read_in(j + 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4_t*>(ct + (lane % 16) * kPitch + i * 16 + 4 * (lane / 16)) = acc[i][j];
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int64_t t = t0 + wm * 64 + j * 16 + p * 8 + tr;
      const float* src = ct + (p * 8 + tr) * kPitch + (lane % 8) * 8;
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(src), hi = *reinterpret_cast<const f32x4_t*>(src + 4);
      float odd[2] = {0.0f, 0.0f};  // NaN where a sum is not finite
      bf16x8_t r;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v0 = q < 2 ? lo[2 * q] : hi[2 * q - 4], v1 = q < 2 ? lo[2 * q + 1] : hi[2 * q - 3];
        odd[0] = __builtin_fmaf(v0, 0.0f, odd[0]);
        odd[1] = __builtin_fmaf(v1, 0.0f, odd[1]);
        r[2 * q] = static_cast<__bf16>(v0 + bf16_lo(own[p][q]));
        r[2 * q + 1] = static_cast<__bf16>(v1 + bf16_hi(own[p][q]));
      }
      const bool on = col && t < T, whole = odd[0] + odd[1] == 0.0f;
      if (on && !whole) again |= 1u << (2 * j + p);
      // dx is not read again here: stored past the caches' replacement order (45 -> 43 us)
      if (on && whole)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, r), reinterpret_cast<u32x4_t*>(dx + t * d + n));
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  // those, in the experts' order (dx_in, which dx may be, still holds what it held)
  for (; again; again &= again - 1) {
    const int b = __builtin_ctz(again);
    const int64_t t = t0 + wm * 64 + b / 2 * 16 + b % 2 * 8 + tr;
    float sum[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] = 0.0f;
#pragma unroll 8
    for (int e = 0; e < E; ++e) {
      const float a = g.dl[t * E + e];
      const u32x4_t u = *reinterpret_cast<const u32x4_t*>(g.wg + e * d + n);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sum[2 * q] = __builtin_fmaf(a, bf16_lo(u[q]), sum[2 * q]);
        sum[2 * q + 1] = __builtin_fmaf(a, bf16_hi(u[q]), sum[2 * q + 1]);
      }
    }
    u32x4_t old = {0, 0, 0, 0};
    if (dx_in) old = *reinterpret_cast<const u32x4_t*>(dx_in + t * d + n);
    bf16x8_t r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      r[2 * q] = static_cast<__bf16>(sum[2 * q] + bf16_lo(old[q]));
      r[2 * q + 1] = static_cast<__bf16>(sum[2 * q + 1] + bf16_hi(old[q]));
    }
    *reinterpret_cast<u32x4_t*>(dx + t * d + n) = __builtin_bit_cast(u32x4_t, r);
  }
}

// Two forms. Up to 64 experts, and for short batches: dWg in 64 x 256 tiles of four
// waves (x streamed once up to 64 experts, the padding experts' products are cheap
// beside it) in one launch with dx and dbias, whose loads and products fill each
// other's waits. Else dWg in 128 x 256 tiles of eight waves, and dx behind it.
constexpr int kColsW = 256, kStagesW = 3, kStagesX = 2;
__global__ __launch_bounds__(512, 1) void dwg_kernel(GateArgs g) {
  typedef DwgTile<128, kColsW, kStagesW> Tile;
  __shared__ __attribute__((aligned(1024))) char lds[Tile::kLds];
  Tile::run(g, blockIdx.x, lds);
}
__global__ __launch_bounds__(256) void gate_dx_kernel(GateArgs g, SumArgs sum) {
  typedef DxTile<kStagesX> Tile;
  __shared__ __attribute__((aligned(1024))) char lds[Tile::kLds];
  const int id = blockIdx.x;
  if (id < g.x_tiles)
    Tile::run(g, id, lds);
  else
    sum_group(sum, id - g.x_tiles, g.E, lds);
}
// dWg, dx and dbias (two stages of both tiles leave room for two workgroups on a CU).
__global__ __launch_bounds__(256) void gate_both_kernel(GateArgs g, SumArgs sum) {
  typedef DwgTile<64, kColsW, 2> W;
  typedef DxTile<kStagesX> X;
  __shared__ __attribute__((aligned(1024))) char lds[W::kLds > X::kLds ? W::kLds : X::kLds];
  const int id = blockIdx.x;
  if (id < g.w_tiles)
    W::run(g, id, lds);
  else if (id < g.w_tiles + g.x_tiles)
    X::run(g, id - g.w_tiles, lds);
  else
    sum_group(sum, id - g.w_tiles - g.x_tiles, g.E, lds);
}

// Batches that take the 64-expert tiles whatever E is: one launch against dWg's
// and dx's, in us, captured, 256 experts at d = 7168: 12.0 / 19.0 at 32 tokens,
// 15.7 / 31.1 at 256, 23.0 / 31.9 at 512; at d = 1024 19.6 / 24.8 at 512 and 30.8 /
// 28.0 at 1024. Up to 64 experts one launch was always the shorter: 2047 x 6144 x
// 16 21.7 / 23.5, 8192 x 4096 x 64 47.9 / 50.5, 300 x 7168 x 64 14.9 / 18.0.
// 65 to 128 experts at more than 512 tokens take the two, and would be shorter in one
// as well: 513 x 7168 x 96 20.2 / 25.6, 1024 x 2048 x 128 18.7 / 25.4, 8192 x 2048 x 65
// 36.5 / 40.1, 4096 x 7168 x 128 54.2 / 62.7.
bool one_launch(int64_t T, int E) { return E <= 64 || T <= 512; }

// Token parts of dWg, at least four steps to each: those of the least estimated
// time, rounds of 256 workgroups (one to a CU) times a part's steps, plus each
// part's way through memory (bytes written and read again). A step takes 1.4 us in
// tiles of 128 experts, 0.8 of 64, a tile's start and end 3; beside the 64-expert
// tiles the parts' sum is a launch of its own, 4. As many parts as one round takes
// are mostly the best (4 for the 56 tiles of 7168 x 256); 4096 x 8448 x 512 with its
// 132 tiles took 229 us in one part and takes 198 in three.
int token_parts(int64_t tiles, int steps, int bm, double bytes) {
  const int64_t most = steps / 4, round = 256 / tiles;
  if (round >= 64) return static_cast<int>(most < 1 ? 1 : most < round ? most : round);
  const double step = bm == 128 ? 1.4 : 0.8, through = bytes / 5.3e6, launch = bm == 128 ? 0.0 : 4.0;
  int best = 1;
  double least = 0.0;
  for (int p = 1; p <= 64 && (p == 1 || p <= most); ++p) {
    const double rounds = static_cast<double>((tiles * p + 255) / 256);
    const double us = rounds * ((steps + p - 1) / p * step + 3.0) + (p > 1 ? launch + p * through : 0.0);
    if (p == 1 || us < least) best = p, least = us;
  }
  return best;
}

__global__ __launch_bounds__(256) void gate_sum_kernel(SumArgs sum, int E) {
  __shared__ __attribute__((aligned(16))) char lds[256 * 8];
  sum_group(sum, sum.bias_groups + blockIdx.x, E, lds);
}

struct GateWs {
  int64_t blocks;
  int bm;
  float* bpart;
  GateArgs g;
};

size_t layout(int64_t T, int64_t d, int E, void* ws, float* dwg, GateWs* w) {
  auto at = [&](size_t off) { return ws ? static_cast<char*>(ws) + off : nullptr; };
  auto pad = [](size_t v) { return (v + 255) / 256 * 256; };
  GateArgs& g = w->g;
  w->bm = one_launch(T, E) ? 64 : 128;
  g.T = T, g.d = d, g.E = E;
  g.Ep = static_cast<int>(up(E, w->bm));
  g.Tp = up(T, kRowsX);
  w->blocks = g.Tp / kBlk;
  g.steps = static_cast<int>((T + kStep - 1) / kStep);
  g.etiles = g.Ep / w->bm;
  const int64_t tiles = (d + kColsW - 1) / kColsW * g.etiles;
  g.parts = token_parts(tiles, g.steps, w->bm, 8.0 * E * d);
  g.w_tiles = static_cast<int>(tiles * g.parts);
  g.ncols = static_cast<int>((d + kColsX - 1) / kColsX);
  g.x_tiles = static_cast<int>(g.ncols * (g.Tp / kRowsX));
  size_t off = 0;
  g.rows = reinterpret_cast<bf16_t*>(at(off));  // [Ep / 32][2][Tp][32]
  off += pad(size_t(2) * g.Tp * g.Ep * 2);
  g.cols = reinterpret_cast<bf16_t*>(at(off));  // [Tp / 32][3][Ep][32]
  off += pad(size_t(3) * g.Tp * g.Ep * 2);
  w->bpart = reinterpret_cast<float*>(at(off));
  off += pad(size_t(w->blocks) * E * 4);
  g.out = dwg;
  if (g.parts > 1) {
    g.out = reinterpret_cast<float*>(at(off));
    off += pad(size_t(g.parts) * E * d * 4);
  }
  return off;
}

}  // namespace

size_t gate_backward_ws(int64_t T, int64_t d, int E) {
  GateWs w{};
  return layout(T, d, E, nullptr, nullptr, &w);
}

hipError_t launch_gate_backward(const void* x, const void* wg, const float* dlogits, const void* dx_in, void* dx,
                                float* dwg, float* dbias, int64_t T, int64_t d, int E, void* ws, hipStream_t s) {
  GateWs w{};
  layout(T, d, E, ws, dwg, &w);
  GateArgs& g = w.g;
  g.x = static_cast<const bf16_t*>(x);
  g.wg = static_cast<const bf16_t*>(wg);
  g.dx_in = static_cast<const bf16_t*>(dx_in);
  g.dl = dlogits;
  g.dx = static_cast<bf16_t*>(dx);
  hipLaunchKernelGGL(split_kernel, dim3(g.Ep / kBlk, static_cast<unsigned>(w.blocks)), dim3(256), 0, s, dlogits, T, E,
                     g.Tp, g.Ep, const_cast<bf16_t*>(g.rows), const_cast<bf16_t*>(g.cols), w.bpart);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  SumArgs sum{};
  sum.part = g.out;
  sum.parts = g.parts;
  sum.n4 = static_cast<int64_t>(E) * d / 4;
  sum.dwg = dwg;
  sum.bpart = w.bpart;
  sum.blocks = static_cast<int>(w.blocks);
  sum.dbias = dbias;
  sum.bias_groups = (E + 15) / 16;
  const int64_t want = (sum.n4 + 255) / 256;
  sum.groups = sum.bias_groups + (g.parts > 1 ? static_cast<int>(want < 2048 ? want : 2048) : 0);
  if (w.bm == 64) {
    hipLaunchKernelGGL(gate_both_kernel, dim3(g.w_tiles + g.x_tiles + sum.bias_groups), dim3(256), 0, s, g, sum);
    if (g.parts == 1) return hipGetLastError();
    if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
    hipLaunchKernelGGL(gate_sum_kernel, dim3(sum.groups - sum.bias_groups), dim3(256), 0, s, sum, E);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(dwg_kernel, dim3(g.w_tiles), dim3(512), 0, s, g);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  hipLaunchKernelGGL(gate_dx_kernel, dim3(g.x_tiles + sum.groups), dim3(256), 0, s, g, sum);
  return hipGetLastError();
}

}  // namespace moe
