// Linear with 4-bit weights and group scales (W4A16):
//
//   out[m, n] = bf16( sum_g s[n, g] * sum_{k in g} x[m, k] * (q[n, k] - z[n, g]) + bias[n] )
//
// q: unsigned 4-bit codes, two per byte; one scale and (optionally) one 4-bit zero point per group
// of G = 32, 64 or 128 elements of a row; without zero points z = 8.
//
// Arithmetic.  Codes become bf16 by bit pattern: 0x3b80 | q is c = 2^-8 (1 + q / 128), exactly.  So a
// group's matrix product gives P = sum x c, and with X = sum 2^-8 x over the group
//   2^-15 sum x (q - z) = P - (1 + z / 128) X,
// X coming from the same matrix instruction against a column of 2^-8.  All of it is exact up to
// fp32 accumulation; the scale multiplies the group's fp32 sum, so no weight is ever rounded, and the
// last step multiplies by 2^15.  The 2^-8 is there for large x: a group of 128 of bf16's largest
// value sums to less than fp32's largest, where with 0x4300 | q (128 + q) a single x of 2.4e36 overflowed
// P and X and their difference was no number.
//
// Tiles: BM = 16 MT rows x BN = 64 CG columns per workgroup of four waves, each wave all rows of
// its 16 CG columns.  Activations go through a ring of NS LDS stages (128 columns each, filled by
// direct global-to-LDS copies, 16-byte chunks XOR-swizzled by row); weights, scales and zero
// points go straight to registers, requested as many steps ahead; once in a turn of NS steps the compiled
// code waits for every request, so on average less is in flight.  Where tiles are few, K is cut into chunks
// whose fp32 partial sums are added in chunk order by launch_dense_split_sum.  Up to four rows take
// a dot-product kernel instead, prompts large tiles over x and scales laid out for them.
#include <algorithm>

#include "layer.hpp"
#include "lds_dma.hpp"

namespace mxq {

namespace {

// bf16 pairs: 2^-8 (1 + q / 128) with q in the low bits; 2^-8.
constexpr uint32_t kI4Code = 0x3b803b80u, kI4One = 0x3b803b80u;
constexpr float kI4Unit = 32768.f;  // sums are kept in units of 2^-15
constexpr int kI4Threads = 256;
constexpr int kI4Stages = 3;
constexpr int kI4DotRows = 4;
// Large tiles: 32-bit offsets within a row tile, one thread per 16 bytes of x in one grid dimension.
constexpr int64_t kI4BigMaxK = 1 << 22, kI4BigMaxX = int64_t(1) << 34;
constexpr int kI4Batch = 4, kI4MaxBatches = 16;
constexpr int64_t kI4DotMaxK = 16384;  // eight waves of 64 blocks

// Eight codes of a dword (element 0 in the lowest nibble) -> eight bf16 2^-8 (1 + q / 128).
__device__ __forceinline__ i32x4 decode8(uint32_t v) {
  const uint32_t e = v & 0x0f0f0f0fu, o = (v >> 4) & 0x0f0f0f0fu;
  i32x4 r;
  r[0] = int(__builtin_amdgcn_perm(o, e, 0x0c040c00u) | kI4Code);
  r[1] = int(__builtin_amdgcn_perm(o, e, 0x0c050c01u) | kI4Code);
  r[2] = int(__builtin_amdgcn_perm(o, e, 0x0c060c02u) | kI4Code);
  r[3] = int(__builtin_amdgcn_perm(o, e, 0x0c070c03u) | kI4Code);
  return r;
}

// Transpose of four dwords over the four 16-lane rows of a wave: dword i of row r goes to dword r
// of row i.
__device__ __forceinline__ i32x4 transpose_rows(const i32x4& d) {
  const auto a = __builtin_amdgcn_permlane32_swap(uint32_t(d[0]), uint32_t(d[2]), false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(uint32_t(d[1]), uint32_t(d[3]), false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return i32x4{int(c[0]), int(c[1]), int(e[0]), int(e[1])};
}

// 1 + z / 128 of a zero point, by its bits or by conversion: the same number, but the tile kernel's schedules
// differ.  us by bits / by conversion, groups of 128: tiles of 16 rows 18.6 / 17.1 (16 x 4096 -> 16384)
// and 26.2 / 24.3 (32 rows); of 64 rows 27.1 / 29.1 (64 x 4096 -> 16384) and 22.0 / 24.9 (128 x 2048 -> 7168).
__device__ __forceinline__ float zero_value(uint32_t z) { return __uint_as_float(0x3f800000u | z << 16); }
template <int MT>
__device__ __forceinline__ float zero_value(uint32_t z) {
  return MT == 1 ? float(128u + z) * 0.0078125f : zero_value(z);
}

// Scale i as loaded (bf16 bits or fp32 bits: nothing is done to it here, so no read has to be waited
// for where it is requested), and its value.
template <bool SBF>
__device__ __forceinline__ uint32_t scale_bits(const void* s, int64_t i) {
  return SBF ? uint32_t(reinterpret_cast<const uint16_t*>(s)[i]) : reinterpret_cast<const uint32_t*>(s)[i];
}
template <bool SBF>
__device__ __forceinline__ float scale_value(uint32_t v) {
  return __uint_as_float(SBF ? v << 16 : v);
}

// Two bf16 products added to c.
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
}

// The value of the lane N places on in this lane's row of 16.
template <int N>
__device__ __forceinline__ float rotate16(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xf, 0xf, true));
}

}  // namespace

// ---------------------------------------------------------------- up to four rows: dot products

// Few rows are bound by reading the weights once, and on one row tile of 16 most of the matrix
// instruction's rows would be empty, so here a lane keeps 32 columns of every x row in registers
// and takes the same 32 columns of weight rows (one 16-byte read each, whole 1 KB pieces of a row
// per wave) through V_DOT2_F32_BF16.  Codes pair up four apart (code i and i + 4 of a dword sit 16
// bits apart, so one AND-OR makes two bf16), x is paired the same way once.  A lane's
// columns lie in one group: its P, less (1 + z / 128) times its X, times the scale, is what the
// wave adds up.  A batch is four weight rows, in two sets of registers; the reads of a next batch hang on
// there being one, and the compiled waits, which have to hold without it too, are for all reads, so
// one batch is on its way at a time.  A batch's sums are reduced over the lanes together, halving rows
// and lanes at once (permlane swaps), and the KW waves of a workgroup, which split K, meet in LDS at the
// end.
//
// LPR lanes hold a row's share (64, or 32 / 16 where the share is that short: a read then covers
// two / four rows).
template <int M, int LPR, bool ZERO, bool SBF>
__global__ __launch_bounds__(512) void int4_dot_kernel(Int4Args a, int kw, int bpw, int batches) {
  constexpr int RB = kI4Batch, NI = RB * LPR / 64;  // rows of a batch, reads of a lane
  __shared__ float part[8][RB * kI4MaxBatches][M];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rows = RB * batches;  // of this workgroup
  const int64_t n0 = int64_t(blockIdx.x) * rows;
  const int K = int(a.K), nblk = K / 32;
  // this lane's block of 32 columns (past the wave's share: none, its x are zeros)
  const int lb = lane & (LPR - 1), blk = wave * bpw + lb;
  const bool on = lb < bpw && blk < nblk;
  const int cb = on ? blk : 0;
  const int gi = cb / (a.group / 32), ngrp = K / a.group, zrow = (ngrp + 1) / 2;
  // the row of this lane's read i: the odd 16-lane rows and the upper half lanes further on where a
  // read covers several
  const int lrow = (LPR <= 32 ? (RB / 2) * (lane >> 5) : 0) + (LPR <= 16 ? (RB / 4) * ((lane >> 4) & 1) : 0);

  struct Batch {
    i32x4 w[NI];
    uint32_t s[NI], z[NI];
  };
  auto load = [&](Batch& o, int b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t n = min<int64_t>(n0 + b * RB + lrow + i, a.N - 1);
      o.w[i] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(a.W + n * (K / 2) + cb * 16));
      o.s[i] = scale_bits<SBF>(a.s, n * ngrp + gi);
      if (ZERO) o.z[i] = a.z[n * zrow + (gi >> 1)];
    }
  };
  Batch even, odd;
  load(even, 0);
  uint32_t x[M][16];
  float xs[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const i32x4* xp = reinterpret_cast<const i32x4*>(reinterpret_cast<const uint16_t*>(a.A) + m * a.lda + cb * 32);
    float t = 0.f;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const i32x4 v = on ? xp[d] : i32x4{0, 0, 0, 0};
      x[m][4 * d + 0] = __builtin_amdgcn_perm(uint32_t(v[2]), uint32_t(v[0]), 0x05040100u);
      x[m][4 * d + 1] = __builtin_amdgcn_perm(uint32_t(v[2]), uint32_t(v[0]), 0x07060302u);
      x[m][4 * d + 2] = __builtin_amdgcn_perm(uint32_t(v[3]), uint32_t(v[1]), 0x05040100u);
      x[m][4 * d + 3] = __builtin_amdgcn_perm(uint32_t(v[3]), uint32_t(v[1]), 0x07060302u);
#pragma unroll
      for (int j = 0; j < 4; ++j) t = dot2(x[m][4 * d + j], kI4One, t);
    }
    xs[m] = t;
  }
  auto compute = [&](const Batch& o, int b) __attribute__((always_inline)) {
    float v[M][NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float acc[M];
#pragma unroll
      for (int m = 0; m < M; ++m) acc[m] = 0.f;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t c = ((uint32_t(o.w[i][d]) >> (4 * j)) & 0x000f000fu) | kI4Code;
#pragma unroll
          for (int m = 0; m < M; ++m) acc[m] = dot2(c, x[m][4 * d + j], acc[m]);
        }
      const float zc = zero_value(ZERO ? (o.z[i] >> (4 * (gi & 1))) & 15u : 8u), s = scale_value<SBF>(o.s[i]);
#pragma unroll
      for (int m = 0; m < M; ++m) v[m][i] = fmaf(-zc, xs[m], acc[m]) * s;
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if constexpr (LPR == 64) {
#pragma unroll
        for (int i = 0; i < RB / 2; ++i) {
          const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[m][i]), __float_as_uint(v[m][i + RB / 2]), false, false);
          v[m][i] = __uint_as_float(t[0]) + __uint_as_float(t[1]);
        }
      }
      if constexpr (LPR >= 32) {
#pragma unroll
        for (int i = 0; i < RB / 4; ++i) {
          const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[m][i]), __float_as_uint(v[m][i + RB / 4]), false, false);
          v[m][i] = __uint_as_float(t[0]) + __uint_as_float(t[1]);
        }
      }
      // the 16 lanes of a row: rotations by 8, 4, 2, 1
#pragma unroll
      for (int i = 0; i < RB / 4; ++i) {
        v[m][i] += rotate16<8>(v[m][i]);
        v[m][i] += rotate16<4>(v[m][i]);
        v[m][i] += rotate16<2>(v[m][i]);
        v[m][i] += rotate16<1>(v[m][i]);
        // every lane of the row holds the sum of weight row i + RB / 4 * (odd row) + RB / 2 * (upper half)
        if ((lane & 15) == i) part[wave][b * RB + i + RB / 4 * ((lane >> 4) & 1) + RB / 2 * (lane >> 5)][m] = v[m][i];
      }
    }
  };
  for (int b = 0; b < batches; b += 2) {
    if (b + 1 < batches) load(odd, b + 1);
    compute(even, b);
    if (b + 2 < batches) load(even, b + 2);
    if (b + 1 < batches) compute(odd, b + 1);
  }
  __syncthreads();
  for (int c = tid; c < rows * M; c += blockDim.x) {
    const int m = c / rows, r = c - m * rows;
    const int64_t n = n0 + r;
    if (n >= a.N) continue;
    float t = 0.f;
    for (int k = 0; k < kw; ++k) t += part[k][r][m];
    float bias = 0.f;
    if (a.bias)
      bias = a.bias_bf16 ? bf16f(reinterpret_cast<const uint16_t*>(a.bias)[n]) : reinterpret_cast<const float*>(a.bias)[n];
    reinterpret_cast<uint16_t*>(a.out)[m * a.ldo + n] = f2bf(fmaf(t, kI4Unit, bias));
  }
}

// ---------------------------------------------------------------- more rows: matrix tiles

// WIDE: a step's scales of a column are read at once, and its zero points, which needs whole steps
// (K % 128 == 0) and aligned pointers.  The reads of 16 columns' rows are what small tiles spend
// their time on: 16 x 7168 -> 2048, groups of 32, 12.0 us against 15.3 with a read each,
// 512 x 7168 -> 2048 56 against 77.
template <int G, int MT, int CG, bool ZERO, bool SBF, bool WIDE>
__global__ __launch_bounds__(kI4Threads) void int4_tile_kernel(Int4Args a) {
  constexpr int NS = kI4Stages, BM = 16 * MT, BN = 64 * CG, STAGE = BM * 256;
  constexpr int GPS = 128 / G;  // groups per step
  constexpr int MPG = G / 32;   // matrix instructions per group
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * BN, m0 = int64_t(blockIdx.y) * BM;
  const int K = int(a.K), ngrp = K / G, zrow = (ngrp + 1) / 2;
  const int nsteps = (K + 127) / 128;
  const int st_b = int(blockIdx.z) * a.split_steps, st_e = min(nsteps, st_b + a.split_steps);
  if (st_b >= st_e) return;  // (the host never cuts K that way)

  // ---- activation copies: this lane's 16-byte slot of each copy, its row and source chunk
  const uint32_t lds0 = lds_addr(smem);
  const uint16_t* asrc[MT];
  int achunk;
  {
    const int r4 = lane >> 4, slot = lane & 15;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = (i * 4 + wave) * 4 + r4;
      asrc[i] = reinterpret_cast<const uint16_t*>(a.A) + min<int64_t>(m0 + row, a.M - 1) * a.lda;
    }
    achunk = slot ^ ((wave * 4 + r4) & 15);  // (row % 16 does not depend on i)
  }
  auto copy = [&](int st, int stage) __attribute__((always_inline)) {
    int c = st * 128 + achunk * 8;
    if (c >= K) c = 0;  // past the row's end: never multiplied
#pragma unroll
    for (int i = 0; i < MT; ++i)
      lds_dma16(asrc[i] + c, lds0 + uint32_t(stage * STAGE + (i * 4 + wave) * 1024));
  };

  // ---- weights
  const uint8_t* wrow[CG];
  int64_t col[CG];
#pragma unroll
  for (int c = 0; c < CG; ++c) {
    col[c] = min<int64_t>(n0 + (wave * CG + c) * 16 + l16, a.N - 1);
    wrow[c] = a.W + col[c] * (K / 2);
  }
  struct Slot {
    i32x4 w[CG];
    uint32_t s[CG][GPS];  // fp32 bits, or a bf16 as loaded (WIDE: two in a word)
    uint32_t z[CG][GPS];  // the byte that holds the zero point (WIDE: the first holds the step's)
  };
  Slot ring[NS];
  auto load = [&](int st, Slot& o) __attribute__((always_inline)) {
    int b = st * 64 + q * 16;
    if (b >= K / 2) b = 0;
#pragma unroll
    for (int c = 0; c < CG; ++c) {
      o.w[c] = *reinterpret_cast<const i32x4*>(wrow[c] + b);
      if constexpr (WIDE) {
        constexpr int B = GPS * (SBF ? 2 : 4);
        __builtin_memcpy(o.s[c], __builtin_assume_aligned(reinterpret_cast<const uint8_t*>(a.s) + col[c] * ngrp * (B / GPS) + st * B, B), B);
        if (GPS == 4) o.z[c][0] = ZERO ? uint32_t(*reinterpret_cast<const uint16_t*>(a.z + col[c] * zrow + st * 2)) : 0x8888u;
        else o.z[c][0] = ZERO ? uint32_t(a.z[col[c] * zrow + st]) : 0x88u;
        continue;
      }
#pragma unroll
      for (int j = 0; j < GPS; ++j) {
        const int g = min(st * GPS + j, ngrp - 1);
        o.s[c][j] = scale_bits<SBF>(a.s, col[c] * ngrp + g);
        o.z[c][j] = ZERO ? uint32_t(a.z[col[c] * zrow + (g >> 1)]) : 0x88u;
      }
    }
  };

  f32x4 acc[MT][CG];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < CG; ++c) acc[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  const i32x4 ones = {int(kI4One), int(kI4One), int(kI4One), int(kI4One)};
  auto compute = [&](int st, const Slot& v, int stage) __attribute__((always_inline)) {
    const uint8_t* as = smem + stage * STAGE + l16 * 256;
    const int blocks = min(4, (K - st * 128) / 32);
    i32x4 wt[CG];
#pragma unroll
    for (int c = 0; c < CG; ++c) wt[c] = G == 128 ? v.w[c] : transpose_rows(v.w[c]);
#pragma unroll
    for (int j = 0; j < GPS; ++j) {
      if (G < 128 && j * MPG >= blocks) break;  // uniform: past the row's end
      i32x4 bf[CG][MPG];
      float s[CG], zc[CG];
#pragma unroll
      for (int c = 0; c < CG; ++c) {
#pragma unroll
        for (int i = 0; i < MPG; ++i) bf[c][i] = decode8(uint32_t(wt[c][j * MPG + i]));
        if (WIDE) {
          s[c] = SBF ? __uint_as_float(j & 1 ? v.s[c][j / 2] & 0xffff0000u : v.s[c][j / 2] << 16) : __uint_as_float(v.s[c][j]);
          zc[c] = zero_value<MT>((v.z[c][0] >> (4 * j)) & 15u);
        } else {
          s[c] = scale_value<SBF>(v.s[c][j]);
          zc[c] = zero_value<MT>((v.z[c][j] >> (4 * ((st * GPS + j) & 1))) & 15u);
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        f32x4 p[CG], x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CG; ++c) p[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < MPG; ++i) {
          // G = 128: instruction i takes dword i of every lane's 32 elements; else 32 elements in a
          // row, eight per lane row
          const int chunk = G == 128 ? 4 * q + i : 4 * (j * MPG + i) + q;
          const i32x4 af = *reinterpret_cast<const i32x4*>(as + mt * 16 * 256 + ((chunk ^ l16) * 16));
#pragma unroll
          for (int c = 0; c < CG; ++c) p[c] = mfma_16x16x32_bf16(af, bf[c][i], p[c]);
          x = mfma_16x16x32_bf16(af, ones, x);
        }
#pragma unroll
        for (int c = 0; c < CG; ++c)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[mt][c][r] = fmaf(fmaf(-zc[c], x[r], p[c][r]), s[c], acc[mt][c][r]);
      }
    }
  };

  // ---- the ring: step st is in stage / slot (st - st_b) % NS; steps past the range repeat the
  // last one and are never computed
#pragma unroll
  for (int u = 0; u < NS - 1; ++u) {
    copy(min(st_b + u, st_e - 1), u);
    load(min(st_b + u, st_e - 1), ring[u]);
  }
  for (int st0 = st_b; st0 < st_e; st0 += NS) {
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      if (st0 + u < st_e) {
        // newer than this step's copies: at least its own weight loads and the next steps' copies and loads
        wait_vmcnt<CG + (NS - 2) * (MT + CG)>();
        __syncthreads();
        const int nx = min(st0 + u + NS - 1, st_e - 1);
        copy(nx, (u + NS - 1) % NS);
        load(nx, ring[(u + NS - 1) % NS]);
        compute(st0 + u, ring[u], u);
      }
    }
  }

  // ---- lane (l16, q) holds rows 4 q + r, column l16 of each 16 x 16 block
  float* const pf = reinterpret_cast<float*>(a.out) + int64_t(blockIdx.z) * a.split_stride;
#pragma unroll
  for (int c = 0; c < CG; ++c) {
    const int64_t n = n0 + (wave * CG + c) * 16 + l16;
    if (n >= a.N) continue;
    float b = 0.f;
    if (a.bias && blockIdx.z == 0)
      b = a.bias_bf16 ? bf16f(reinterpret_cast<const uint16_t*>(a.bias)[n]) : reinterpret_cast<const float*>(a.bias)[n];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t m = m0 + mt * 16 + 4 * q + r;
        if (m >= a.M) continue;
        const float v = fmaf(acc[mt][c][r], kI4Unit, b);
        if (a.splits > 1)
          pf[m * a.N + n] = v;
        else
          reinterpret_cast<uint16_t*>(a.out)[m * a.ldo + n] = f2bf(v);
      }
  }
}

// ---------------------------------------------------------------- many rows: large matrix tiles

// A prompt is bound by the matrix instructions, so everything that is not one is taken out of the
// loop: a pass over x first writes it with the eight columns of every 16-byte chunk in the order
// 0 4 1 5 2 6 3 7 -- the order in which (v & 0x000f000f) | 0x3b803b80 and three shifts of it give
// the codes of a dword, seven instructions for eight codes -- and the groups' sums X.  The
// product of a group starts from -(1 + z / 128) X, so what comes out is 2^-15 sum x (q - z).
__global__ __launch_bounds__(256) void int4_prep_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, int64_t lda,
                                                        int group, int64_t Mp, uint16_t* __restrict__ xp,
                                                        float* __restrict__ X) {
  const int64_t chunks = K / 8, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t m = i / chunks, c = i - m * chunks;
  const int per = group / 8;  // chunks of a group: 4, 8 or 16 neighbouring lanes (rows are whole groups)
  float t = 0.f;
  if (m < M) {
    const uint4 v = *reinterpret_cast<const uint4*>(x + m * lda + c * 8);
    uint4 o;
    o.x = __builtin_amdgcn_perm(v.z, v.x, 0x05040100u);
    o.y = __builtin_amdgcn_perm(v.z, v.x, 0x07060302u);
    o.z = __builtin_amdgcn_perm(v.w, v.y, 0x05040100u);
    o.w = __builtin_amdgcn_perm(v.w, v.y, 0x07060302u);
    *reinterpret_cast<uint4*>(xp + m * K + c * 8) = o;
    t = dot2(o.x, kI4One, dot2(o.y, kI4One, dot2(o.z, kI4One, dot2(o.w, kI4One, 0.f))));
  }
  for (int o = 1; o < per; o <<= 1) t += __shfl_xor(t, o, kWave);
  if (m < M && (c & (per - 1)) == 0) X[(c / per) * Mp + m] = t;
}

// The scales and zero points as the large tiles take them: (s, -(1 + z / 128)) fp32 pairs, columns
// neighbouring ([group][Np]), so that a step's arrive in LDS with one copy per group: gathered by every
// wave from their rows, they were most of the loop's vector memory instructions.
template <bool ZERO, bool SBF>
__global__ __launch_bounds__(256) void int4_scale_prep_kernel(Int4Args a, int64_t Np, float2* __restrict__ sz) {
  const int ngrp = int(a.K / a.group), zrow = (ngrp + 1) / 2;
  const int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (n >= Np) return;
  const int64_t nc = min<int64_t>(n, a.N - 1);
  for (int g = int(blockIdx.y); g < ngrp; g += int(gridDim.y)) {
    const float s = scale_value<SBF>(scale_bits<SBF>(a.s, nc * ngrp + g));
    const uint32_t z = ZERO ? (uint32_t(a.z[nc * zrow + (g >> 1)]) >> (4 * (g & 1))) & 15u : 8u;
    sz[int64_t(g) * Np + n] = make_float2(s, -zero_value(z));
  }
}

// BM = 256 rows x BN = 128 columns, eight waves of 64 x 64; lane l16 of column group c holds column
// 4 l16 + c of its wave's 64, so a lane ends with four neighbouring columns of each of its rows.
// A stage holds x, codes, group sums and pairs, all copied by DMA a step ahead: 148 to 160 KB for
// two.  (Codes straight to registers, read by each of the four waves that use them, took 107 us
// where this takes 92.)
// Measured: 2048 x 2048 -> 7168 in 89 / 110 / 131 us with groups of 128 / 64 / 32, the passes over x
// and the scales included (128: 674 TFLOP/s); the 64 x 128 and 128 x 128 tiles take 130 / 218 / 316.
// Nothing bounds it alone: a step takes 2.4 us, its matrix instructions 0.9; without the copies it
// is 14 % shorter, without three of four matrix instructions 10 %, without the scales' arithmetic
// 9 %.  The two waves of a SIMD pass the same barrier and so wait together.
constexpr int kBigM = 256, kBigN = 128, kBigThreads = 512;

template <int G>
__global__ __launch_bounds__(kBigThreads, 2) void int4_big_kernel(Int4Args a, const float* __restrict__ X, int64_t Mp,
                                                                  const float2* __restrict__ sz, int64_t Np) {
  constexpr int GPS = 128 / G, MPG = G / 32, MT = 4, CG = 4;
  constexpr int A_BYTES = kBigM * 256, W_BYTES = kBigN * 64, X_BYTES = GPS * kBigM * 4;
  constexpr int W_AT = A_BYTES, X_AT = W_AT + W_BYTES, S_AT = X_AT + X_BYTES, STAGE = S_AT + GPS * kBigN * 8;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int wm = wave & 3, wn = wave >> 2;  // four waves along the rows, two along the columns
  const int64_t n0 = int64_t(blockIdx.x) * kBigN, m0 = int64_t(blockIdx.y) * kBigM;
  const int K = int(a.K), ngrp = K / G, nsteps = (K + 127) / 128;

  const uint32_t lds0 = lds_addr(smem);
  const int r4 = lane >> 4, slot = lane & 15;
  const int achunk = slot ^ ((wave * 4 + r4) & 15);  // (row % 16: 32 i drops out)
  // operands as a uniform base and 32-bit lane offsets (K <= 2^22, so 256 rows stay below 2^31 bytes)
  const uint16_t* const ab = reinterpret_cast<const uint16_t*>(a.A) + m0 * K;
  const int arows = int(min<int64_t>(a.M - m0, kBigM)), ncols = int(min<int64_t>(a.N - n0, kBigN));
  // weights: LDS row 16 (4 wn + c) + l16 is column 64 wn + 4 l16 + c of the tile, its four 16-byte
  // chunks XOR-swizzled by l16 / 4; wave w copies LDS rows [16 w, +16)
  const uint8_t* const wb = a.W + n0 * (K / 2);
  const uint32_t wrow = uint32_t(min((wave >> 2) * 64 + 4 * r4 * 4 + (slot >> 2) * 4 + (wave & 3), ncols - 1)) * uint32_t(K / 2);
  const int wchunk = (slot & 3) ^ r4;
  auto copy = [&](int st, int stage) __attribute__((always_inline)) {
    int c = st * 128 + achunk * 8;
    if (c >= K) c = 0;  // past the row's end: never multiplied
    uint32_t b = uint32_t(st * 64 + wchunk * 16);
    if (b >= uint32_t(K / 2)) b = 0;
    lds_dma16(wb, wrow + b, lds0 + uint32_t(stage * STAGE + W_AT + wave * 1024));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      lds_dma16(ab, uint32_t(min((i * 8 + wave) * 4 + r4, arows - 1) * K + c) * 2u,
                lds0 + uint32_t(stage * STAGE + (i * 8 + wave) * 1024));
    const int g = min(st * GPS + (wave & (GPS - 1)), ngrp - 1);
    if (wave < GPS)  // 256 group sums; 128 scale and zero point pairs
      lds_dma16(X + int64_t(g) * Mp + m0 + lane * 4, lds0 + uint32_t(stage * STAGE + X_AT + wave * (kBigM * 4)));
    else if (wave < 2 * GPS)
      lds_dma16(sz + int64_t(g) * Np + n0 + lane * 2,
                lds0 + uint32_t(stage * STAGE + S_AT + (wave - GPS) * (kBigN * 8)));
  };

  f32x4 acc[MT][CG];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < CG; ++c) acc[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  // One step.  Its codes are turned into bf16 in HALVES parts (a whole group at least).
  constexpr int HALVES = G == 128 ? 1 : 2, FR = 4 / HALVES, HG = GPS / HALVES;  // blocks, groups of a part
  auto step = [&](int st, int stage) __attribute__((always_inline)) {
    const uint8_t* ws = smem + stage * STAGE + W_AT + wn * 4096 + l16 * 64 + ((q ^ (l16 >> 2)) * 16);
    const uint8_t* as = smem + stage * STAGE + (wm * 64 + l16) * 256;
    const uint8_t* xs = smem + stage * STAGE + X_AT + (wm * 64 + 4 * q) * 4;
    const uint8_t* ss = smem + stage * STAGE + S_AT + (wn * 64 + 4 * l16) * 8;
    const int blocks = min(4, (K - st * 128) / 32);
    i32x4 w[CG];
#pragma unroll
    for (int c = 0; c < CG; ++c) {
      w[c] = *reinterpret_cast<const i32x4*>(ws + c * 1024);
      if (G < 128) w[c] = transpose_rows(w[c]);
    }
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      i32x4 bf[CG][FR];
      float s[CG][HG], zc[CG][HG];
#pragma unroll
      for (int c = 0; c < CG; ++c) {
#pragma unroll
        for (int i = 0; i < FR; ++i) {
          const uint32_t u = uint32_t(w[c][h * FR + i]);
#pragma unroll
          for (int d = 0; d < 4; ++d) bf[c][i][d] = int(((u >> (4 * d)) & 0x000f000fu) | kI4Code);
        }
      }
#pragma unroll
      for (int j = 0; j < HG; ++j) {
        const f32x4 p0 = *reinterpret_cast<const f32x4*>(ss + (h * HG + j) * (kBigN * 8));
        const f32x4 p1 = *reinterpret_cast<const f32x4*>(ss + (h * HG + j) * (kBigN * 8) + 16);
        s[0][j] = p0[0]; zc[0][j] = p0[1]; s[1][j] = p0[2]; zc[1][j] = p0[3];
        s[2][j] = p1[0]; zc[2][j] = p1[1]; s[3][j] = p1[2]; zc[3][j] = p1[3];
      }
#pragma unroll
      for (int j = 0; j < HG; ++j) {
        const int g = h * HG + j;  // of the step's groups
        if (G < 128 && g * MPG >= blocks) break;  // uniform: past the row's end
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(xs + g * (kBigM * 4) + mt * 64);
          f32x4 p[CG];
#pragma unroll
          for (int c = 0; c < CG; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) p[c][r] = zc[c][j] * x[r];
#pragma unroll
          for (int i = 0; i < MPG; ++i) {
            const int chunk = G == 128 ? 4 * q + i : 4 * (g * MPG + i) + q;
            const i32x4 af = *reinterpret_cast<const i32x4*>(as + mt * 16 * 256 + ((chunk ^ l16) * 16));
#pragma unroll
            for (int c = 0; c < CG; ++c) p[c] = mfma_16x16x32_bf16(af, bf[c][j * MPG + i], p[c]);
          }
#pragma unroll
          for (int c = 0; c < CG; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[mt][c][r] = fmaf(p[c][r], s[c][j], acc[mt][c][r]);
        }
      }
    }
  };

  copy(0, 0);
  for (int st = 0; st < nsteps; ++st) {
    wait_vmcnt<0>();  // this step's copies, requested a step ago
    __syncthreads();  // and everyone's; the other stage has been read
    if (st + 1 < nsteps) copy(st + 1, (st + 1) & 1);
    step(st, st & 1);
  }

  // ---- lane (l16, q): rows 4 q + r, columns 4 l16 .. + 4
  const int64_t n = n0 + wn * 64 + 4 * l16;
  float b[CG];
#pragma unroll
  for (int c = 0; c < CG; ++c)
    b[c] = !a.bias ? 0.f
                   : a.bias_bf16 ? bf16f(reinterpret_cast<const uint16_t*>(a.bias)[n0 + min(wn * 64 + 4 * l16 + c, ncols - 1)])
                                 : reinterpret_cast<const float*>(a.bias)[n0 + min(wn * 64 + 4 * l16 + c, ncols - 1)];
  const bool whole = n + 4 <= a.N && (a.ldo & 3) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t m = m0 + wm * 64 + mt * 16 + 4 * q + r;
      if (m >= a.M) continue;
      uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + m * a.ldo + n;
      const uint32_t lo = pack_bf16x2(fmaf(acc[mt][0][r], kI4Unit, b[0]), fmaf(acc[mt][1][r], kI4Unit, b[1]));
      const uint32_t hi = pack_bf16x2(fmaf(acc[mt][2][r], kI4Unit, b[2]), fmaf(acc[mt][3][r], kI4Unit, b[3]));
      if (whole) {
        *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
      } else {
        if (n + 0 < a.N) o[0] = uint16_t(lo);
        if (n + 1 < a.N) o[1] = uint16_t(lo >> 16);
        if (n + 2 < a.N) o[2] = uint16_t(hi);
        if (n + 3 < a.N) o[3] = uint16_t(hi >> 16);
      }
    }
}

// ---------------------------------------------------------------- host side

// GO(zero points given, bf16 scales)
#define MXQ_I4_PICK(GO)                         \
  do {                                          \
    if (a.z && a.s_bf16) GO(true, true);        \
    else if (a.z) GO(true, false);              \
    else if (a.s_bf16) GO(false, true);         \
    else GO(false, false);                      \
  } while (0)

namespace {
template <int G, int MT, int CG>
void launch_i4(const Int4Args& a, hipStream_t st) {
  const dim3 grid(unsigned(cdiv(a.N, 64 * CG)), unsigned(cdiv(a.M, 16 * MT)), unsigned(a.splits));
  const size_t lds = size_t(kI4Stages) * MT * 16 * 256;
  if constexpr (G < 128) {
    constexpr int GPS = 128 / G;
    if (a.K % 128 == 0 && reinterpret_cast<uintptr_t>(a.s) % (GPS * (a.s_bf16 ? 2 : 4)) == 0 &&
        reinterpret_cast<uintptr_t>(a.z) % 2 == 0) {
#define MXQ_I4(Z, S) \
  hipLaunchKernelGGL((int4_tile_kernel<G, MT, CG, Z, S, true>), grid, dim3(kI4Threads), lds, st, a)
      MXQ_I4_PICK(MXQ_I4);
#undef MXQ_I4
      return;
    }
  }
#define MXQ_I4(Z, S) \
  hipLaunchKernelGGL((int4_tile_kernel<G, MT, CG, Z, S, false>), grid, dim3(kI4Threads), lds, st, a)
  MXQ_I4_PICK(MXQ_I4);
#undef MXQ_I4
}

template <int G>
void launch_i4_g(const Int4Args& a, const Int4Plan& p, hipStream_t st) {
  if (p.mt == 1) launch_i4<G, 1, 1>(a, st);
  else if (p.mt == 4) launch_i4<G, 4, 2>(a, st);
  else launch_i4<G, 8, 2>(a, st);
}

template <int G>
void launch_i4_big(const Int4Args& a, const float* X, int64_t Mp, const float2* sz, int64_t Np, hipStream_t st) {
  const dim3 grid(unsigned(cdiv(a.N, kBigN)), unsigned(cdiv(a.M, kBigM)));
  const size_t lds = 2 * (size_t(kBigM) * 256 + kBigN * 64 + (128 / G) * (kBigM * 4 + kBigN * 8));
  hipLaunchKernelGGL((int4_big_kernel<G>), grid, dim3(kBigThreads), lds, st, a, X, Mp, sz, Np);
}

template <int M, int LPR>
void launch_dot_z(const Int4Args& a, int kw, int bpw, int batches, hipStream_t st) {
  const dim3 grid(unsigned(cdiv(a.N, kI4Batch * batches))), block(unsigned(64 * kw));
#define MXQ_I4(Z, S) hipLaunchKernelGGL((int4_dot_kernel<M, LPR, Z, S>), grid, block, 0, st, a, kw, bpw, batches)
  MXQ_I4_PICK(MXQ_I4);
#undef MXQ_I4
}

template <int M>
void launch_dot_l(const Int4Args& a, int kw, int bpw, int batches, hipStream_t st) {
  if (bpw <= 16) launch_dot_z<M, 16>(a, kw, bpw, batches, st);
  else if (bpw <= 32) launch_dot_z<M, 32>(a, kw, bpw, batches, st);
  else launch_dot_z<M, 64>(a, kw, bpw, batches, st);
}

// Waves along K (64 blocks of 32 columns each at most), the blocks of a wave, and as many batches
// per workgroup as leave 4096 waves for one row, 2048 for more (their registers leave room for
// eight waves on a compute unit; 4096 x 16384 with groups of 64: one row 13.1 us against 16.5 with
// 2048 waves and 26.7 with 1024, three rows 24.5, 19.0, 31.5 us).
void launch_int4_dot(const Int4Args& a, hipStream_t st) {
  const int nblk = int(a.K / 32);
  const int kw = int(cdiv(nblk, 64)), bpw = int(cdiv(nblk, kw));
  const int batches = int(std::max<int64_t>(1, std::min<int64_t>(kI4MaxBatches, a.N * kw / (kI4Batch * (a.M == 1 ? 4096 : 2048)))));
  switch (a.M) {
    case 1: launch_dot_l<1>(a, kw, bpw, batches, st); break;
    case 2: launch_dot_l<2>(a, kw, bpw, batches, st); break;
    case 3: launch_dot_l<3>(a, kw, bpw, batches, st); break;
    default: launch_dot_l<4>(a, kw, bpw, batches, st); break;
  }
}
}  // namespace

// Workspace of the large tiles: x in its new order, the groups' sums (whole row tiles), the scale and
// zero point pairs (whole column tiles).
struct BigWs {
  int64_t Mp, Np;
  size_t sums, pairs, total;
};
static BigWs int4_big_ws(int64_t M, int64_t N, int64_t K, int group) {
  BigWs w;
  w.Mp = cdiv(M, kBigM) * kBigM;
  w.Np = cdiv(N, kBigN) * kBigN;
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  w.sums = up(size_t(M) * size_t(K) * 2);
  w.pairs = w.sums + up(size_t(K / group) * size_t(w.Mp) * 4);
  w.total = w.pairs + size_t(K / group) * size_t(w.Np) * 8;
  return w;
}

Int4Plan int4_plan(int64_t M, int64_t N, int64_t K, int group) {
  Int4Plan p{};
  p.splits = 1;
  p.split_steps = int32_t(cdiv(K, 128));
  if (M <= kI4DotRows && K <= kI4DotMaxK) return p;
  // The large tiles, once they occupy three of four compute units, or half of them with groups below
  // 128, which cost the other kernel one more product of ones each (us, large tiles against the others:
  // 1024 x 2048 -> 7168, 224 tiles, 60 against 67 with groups of 128, 77 against 160 with 32;
  // 1024 x 4096 -> 4096, 128 tiles, 103 against 66 and 126 against 154; 700 x 7168 -> 4096, 96 tiles,
  // groups of 64, 170 against 172; 512 x 7168 -> 2048, 32 tiles, groups of 32, 207 against 88) -- and the
  // rows fill more than half a tile: on wide weights the grid says nothing about them (K = 4096, groups
  // of 64: 8 rows to N = 16384 102 against 21, 64 to 28672 111 against 49, 128 to 28672 114 against
  // 97, but 160 to 20480 109 against 172; groups of 32, 128 to 28672 144 against 135, 192 146 against
  // 259; groups of 128, 128 to 28672 85 against 62, 160 to 24576 84 against 112).
  if (M > kBigM / 2 && K <= kI4BigMaxK && M <= kI4BigMaxX / K && cdiv(M, kBigM) * cdiv(N, kBigN) >= (group == 128 ? 192 : 128)) {
    p.mt = 16;
    p.partial_bytes = int4_big_ws(M, N, K, group).total;
    return p;
  }
  // Rows of a tile (us with tiles of 16 x 64, 64 x 128, 128 x 128, one read per scale): few workgroups take longer than
  // the weights read again -- 97 x 576 -> 224: 6.2, 15.8, 23.3; 32 x 7168 -> 2048: 16.1, 24.1, -;
  // 64 x 7168 -> 2048: 14.8, 20.2, -; but 64 x 4096 -> 4096, groups of 32: 42.9, 30.0, -;
  // 128 x 2048 -> 7168: 37.3, 29.9, 34.4; 512 x 2048 -> 2048: 37.5, 29.7, 33.9.
  if (M <= 32 || cdiv(M, 16) * cdiv(N, 64) <= 128) p.mt = 1;
  else if (M <= 64 || cdiv(M, 64) * cdiv(N, 128) <= 256) p.mt = 4;
  else p.mt = 8;
  const int cg = p.mt == 1 ? 1 : 2;
  const int64_t tiles = cdiv(N, 64 * cg) * cdiv(M, 16 * p.mt), nsteps = cdiv(K, 128);
  int64_t s = 1;
  // chunks of at least four steps until the grid reaches two workgroups per compute unit, the
  // partial sums at most 16 MiB
  while (s < 8 && tiles * s < 512 && nsteps >= 8 * s && 2 * s * M * N * 4 <= (int64_t(16) << 20)) s *= 2;
  p.split_steps = int32_t(cdiv(nsteps, s));
  p.splits = int32_t(cdiv(nsteps, p.split_steps));
  p.partial_bytes = p.splits > 1 ? size_t(p.splits) * size_t(M) * size_t(N) * 4 : 0;
  return p;
}

void launch_int4_linear(const Int4Args& g, int group, float* partial, hipStream_t stream) {
  if (g.M <= 0 || g.N <= 0) return;
  const Int4Plan p = int4_plan(g.M, g.N, g.K, group);
  Int4Args a = g;
  a.group = group;
  if (p.mt == 0) {
    launch_int4_dot(a, stream);
    return;
  }
  if (p.mt == 16) {
    const BigWs w = int4_big_ws(a.M, a.N, a.K, group);
    uint8_t* base = reinterpret_cast<uint8_t*>(partial);
    uint16_t* xp = reinterpret_cast<uint16_t*>(base);
    float* X = reinterpret_cast<float*>(base + w.sums);
    float2* sz = reinterpret_cast<float2*>(base + w.pairs);
    const int64_t Mp = w.Mp, Np = w.Np;
    const dim3 pg(unsigned(cdiv(a.M * (a.K / 8), 256)));
    hipLaunchKernelGGL(int4_prep_kernel, pg, dim3(256), 0, stream, static_cast<const uint16_t*>(a.A), a.M, a.K, a.lda,
                       group, Mp, xp, X);
    a.A = xp;
    const dim3 sg(unsigned(cdiv(Np, 256)), unsigned(std::min<int64_t>(a.K / group, 256)));
#define MXQ_I4(Z, S) hipLaunchKernelGGL((int4_scale_prep_kernel<Z, S>), sg, dim3(256), 0, stream, a, Np, sz)
    MXQ_I4_PICK(MXQ_I4);
#undef MXQ_I4
    if (group == 32) launch_i4_big<32>(a, X, Mp, sz, Np, stream);
    else if (group == 64) launch_i4_big<64>(a, X, Mp, sz, Np, stream);
    else launch_i4_big<128>(a, X, Mp, sz, Np, stream);
    return;
  }
  a.splits = p.splits;
  a.split_steps = p.split_steps;
  a.split_stride = g.M * g.N;
  if (p.splits > 1) a.out = partial;
  if (group == 32) launch_i4_g<32>(a, p, stream);
  else if (group == 64) launch_i4_g<64>(a, p, stream);
  else launch_i4_g<128>(a, p, stream);
  if (p.splits > 1)
    launch_dense_split_sum(partial, p.splits, g.M, g.N, static_cast<uint16_t*>(g.out), g.ldo, stream);
}

}  // namespace mxq
