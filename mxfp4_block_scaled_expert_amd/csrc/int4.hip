// Linear with 4-bit weights and group scales (W4A16):
//
//   out[m, n] = bf16( sum_g s[n, g] * sum_{k in g} x[m, k] * (q[n, k] - z[n, g]) + bias[n] )
//
// q: unsigned 4-bit codes, two per byte; one scale and (optionally) one 4-bit zero point per group
// of G = 32, 64 or 128 elements of a row; without zero points z = 8.
//
// Arithmetic.  Codes become bf16 by bit pattern: 0x4300 | q is 128 + q, exactly.  So a group's
// matrix product gives sum x (128 + q), and with X = sum x over the group
//   sum x (q - z) = sum x (128 + q) - (128 + z) X,
// X coming from the same matrix instruction against a column of ones.  All of it is exact up to
// fp32 accumulation; the scale multiplies the group's fp32 sum, so no weight is ever rounded.
//
// Tiles: BM = 16 MT rows x BN = 64 CG columns per workgroup of four waves, each wave all rows of
// its 16 CG columns.  Activations go through a ring of NS LDS stages (128 columns each, filled by
// direct global-to-LDS copies, 16-byte chunks XOR-swizzled by row); weights, scales and zero
// points go straight to registers, as many steps ahead.  Where tiles are few, K is cut into chunks
// whose fp32 partial sums are added in chunk order by launch_dense_split_sum.
#include <algorithm>

#include "lds_dma.hpp"
#include "kernels.hpp"

namespace mxq {

namespace {

constexpr int kI4Threads = 256;
constexpr int kI4Stages = 3;

// Eight codes of a dword (element 0 in the lowest nibble) -> eight bf16 128 + q.
__device__ __forceinline__ i32x4 decode8(uint32_t v) {
  const uint32_t e = v & 0x0f0f0f0fu, o = (v >> 4) & 0x0f0f0f0fu;
  i32x4 r;
  r[0] = int(__builtin_amdgcn_perm(o, e, 0x0c040c00u) | 0x43004300u);
  r[1] = int(__builtin_amdgcn_perm(o, e, 0x0c050c01u) | 0x43004300u);
  r[2] = int(__builtin_amdgcn_perm(o, e, 0x0c060c02u) | 0x43004300u);
  r[3] = int(__builtin_amdgcn_perm(o, e, 0x0c070c03u) | 0x43004300u);
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

}  // namespace

template <int G, int MT, int CG>
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
    uint32_t s[CG][GPS];  // fp32 bits, or a bf16 as loaded
    uint32_t z[CG][GPS];  // the byte that holds the zero point
  };
  Slot ring[NS];
  auto load = [&](int st, Slot& o) __attribute__((always_inline)) {
    int b = st * 64 + q * 16;
    if (b >= K / 2) b = 0;
#pragma unroll
    for (int c = 0; c < CG; ++c) {
      o.w[c] = *reinterpret_cast<const i32x4*>(wrow[c] + b);
#pragma unroll
      for (int j = 0; j < GPS; ++j) {
        const int g = min(st * GPS + j, ngrp - 1);
        o.s[c][j] = a.s_bf16 ? uint32_t(reinterpret_cast<const uint16_t*>(a.s)[col[c] * ngrp + g])
                             : reinterpret_cast<const uint32_t*>(a.s)[col[c] * ngrp + g];
        o.z[c][j] = a.z ? uint32_t(a.z[col[c] * zrow + (g >> 1)]) : 0x88u;
      }
    }
  };

  f32x4 acc[MT][CG];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < CG; ++c) acc[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  const i32x4 ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
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
        s[c] = a.s_bf16 ? bf16f(uint16_t(v.s[c][j])) : __uint_as_float(v.s[c][j]);
        const int g = st * GPS + j;
        zc[c] = float(128u + ((v.z[c][j] >> (4 * (g & 1))) & 15u));
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
        const float v = acc[mt][c][r] + b;
        if (a.splits > 1)
          pf[m * a.N + n] = v;
        else
          reinterpret_cast<uint16_t*>(a.out)[m * a.ldo + n] = f2bf(v);
      }
  }
}

// ---------------------------------------------------------------- host side

namespace {
template <int G, int MT, int CG>
void launch_i4(const Int4Args& a, hipStream_t st) {
  const dim3 grid(unsigned(cdiv(a.N, 64 * CG)), unsigned(cdiv(a.M, 16 * MT)), unsigned(a.splits));
  hipLaunchKernelGGL((int4_tile_kernel<G, MT, CG>), grid, dim3(kI4Threads), size_t(kI4Stages) * MT * 16 * 256, st, a);
}

template <int G>
void launch_i4_g(const Int4Args& a, const Int4Plan& p, hipStream_t st) {
  if (p.mt == 1) launch_i4<G, 1, 1>(a, st);
  else if (p.mt == 4) launch_i4<G, 4, 2>(a, st);
  else launch_i4<G, 8, 2>(a, st);
}
}  // namespace

Int4Plan int4_plan(int64_t M, int64_t N, int64_t K) {
  Int4Plan p{};
  p.mt = M <= 16 ? 1 : (M <= 64 ? 4 : 8);
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
  const Int4Plan p = int4_plan(g.M, g.N, g.K);
  Int4Args a = g;
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
