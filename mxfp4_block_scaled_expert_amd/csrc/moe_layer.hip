// A whole routed-expert layer for a few tokens: router product, routing, gate/up, SiLU-and-mul,
// down and the weighted sum over each token's experts, in three launches and without a sort.
//
//   logits[t, e] = sum_k x[t, k] gate[e, k] + gate_bias[e]              (fp32)
//   (ids, w)     = the routing of route_common.hpp
//   h[t, j]      = w[t, j] * silu(g) * u,  [g | u] = x[t] @ w1[e]^T + b1[e],  e = ids[t, j]
//   out[t]       = bf16( sum_j h[t, j] @ w2[ids[t, j]]^T )
//
// What bounds it: reading the chosen experts' weights once (a token of a 128-expert MXFP4 layer
// with H = I = 2880 and top-4: 53 MB; of a 256-expert FP8 layer with H = 7168, I = 2048, top-8:
// 352 MB), and for one token the latency of three dependent launches.  So both expert stages are
// weight streams: every wave keeps a D-deep ring of 128-byte row steps in flight in registers, the
// ring running on across its work items, and the activations come from LDS, so that no other
// vector memory read gets between the stream's waits.
//
//  * moe_gate_kernel: the router product on V_MFMA_F32_16X16X32_BF16, split over experts and K;
//    fp32 router weights are split into three bf16 terms that sum to them exactly.  Partial sums
//    go to the workspace and are added in order where they are read.
//  * moe_up_kernel: every workgroup routes all tokens itself (one wave per token: the logits are
//    a few KB) and builds the same tables in LDS: chosen experts ascending, each with its rows
//    (tokens ascending).  A wave's item is 16 gate columns and the 16 matching up columns of one
//    expert over the whole K, so its epilogue has both halves in registers.
//  * moe_down_kernel: a workgroup's item is 16 output columns over ALL chosen experts; its eight
//    waves split the (expert rows, K steps) evenly, and their sums meet in LDS, each token's rows
//    added in a fixed order -- no partial outputs in memory, no atomics, no combine launch.  The
//    rows of h are copied into LDS in batches of B sorted rows, one batch ahead.
//
// Rounding: products and sums are fp32.  The routing weight joins h in fp32.  h is kept as two
// bf16 terms (hi + lo, relative error 2^-17 of it): with one bf16 term the output's error against
// 64 bits would be 1.4 times its own rounding.  The 16 rows of the MFMA are mostly empty here, so
// hi and lo are simply two rows of the same product.
#include <algorithm>

#include "lds_dma.hpp"
#include "kernels.hpp"
#include "route_common.hpp"

namespace mxq {

namespace {
constexpr int kLyThreads = 512, kLyWaves = 8;
constexpr int kGateThreads = 256;
constexpr int kUpD = 4;    // ring depth of the gate/up stream: 3 steps of 4 KB per wave in flight
constexpr int kDownD = 8;  // of the down stream: 7 steps of 2 KB
}  // namespace

// ---------------------------------------------------------------- router product

// part[s][t][e]: the sum over K chunk s.  Grid: (ceil(E / 16), S); the four waves of a workgroup
// take the chunk's 32-wide steps in turn.
template <bool F32W>
__global__ __launch_bounds__(kGateThreads) void moe_gate_kernel(const uint16_t* __restrict__ x, int32_t M, int64_t ldx,
                                                                const void* __restrict__ gate, int32_t E, int64_t H,
                                                                int32_t chunk, float* __restrict__ part) {
  __shared__ float red[4][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, q = lane >> 4;
  const int e0 = int(blockIdx.x) * 16;
  const int k0 = int(blockIdx.y) * chunk, k1 = min(int(H), k0 + chunk);
  const uint16_t* xr = x + int64_t(min(l16, M - 1)) * ldx + q * 8;
  const int64_t grow = int64_t(min(e0 + l16, E - 1)) * H + q * 8;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int k = k0 + wave * 32; k < k1; k += 128) {
    const i32x4 af = *reinterpret_cast<const i32x4*>(xr + k);
    if constexpr (F32W) {
      const float* gp = reinterpret_cast<const float*>(gate) + grow + k;
      const f32x4 g0 = *reinterpret_cast<const f32x4*>(gp), g1 = *reinterpret_cast<const f32x4*>(gp + 4);
      float v[8] = {g0[0], g0[1], g0[2], g0[3], g1[0], g1[1], g1[2], g1[3]};
      // v = t0 + t1 + t2 with bf16 terms: each term takes the next eight bits of the significand
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        i32x4 b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = pack_bf16x2(v[2 * i], v[2 * i + 1]);
          b[i] = int(w);
          // (an infinite or NaN weight has no remainder)
          const float lo = bf16lo(w), hi = bf16hi(w);
          v[2 * i] = fabsf(lo) < __builtin_huge_valf() ? v[2 * i] - lo : 0.f;
          v[2 * i + 1] = fabsf(hi) < __builtin_huge_valf() ? v[2 * i + 1] - hi : 0.f;
        }
        acc = mfma_16x16x32_bf16(af, b, acc);
      }
    } else {
      const i32x4 bf = *reinterpret_cast<const i32x4*>(reinterpret_cast<const uint16_t*>(gate) + grow + k);
      acc = mfma_16x16x32_bf16(af, bf, acc);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) red[wave][4 * q + r][l16] = acc[r];
  __syncthreads();
  const int t = tid >> 4, e = tid & 15;
  if (t < M && e0 + e < E)
    part[(int64_t(blockIdx.y) * M + t) * E + e0 + e] = (red[0][t][e] + red[1][t][e]) + (red[2][t][e] + red[3][t][e]);
}

// ---------------------------------------------------------------- routing tables in LDS

struct LayerTables {
  int32_t* mask;    // [E] tokens of each expert, one bit per token
  int32_t* start;   // [E] first sorted row of each expert
  int32_t* touch;   // [E] chosen experts, ascending
  int32_t* id;      // [R] expert of flat row t * topk + k
  float* w;         // [R]
  int32_t* row;     // [R] sorted rows: expert << 8 | token
  float* roww;      // [R] their routing weights
  int32_t* seg;     // [R] segments: runs of one expert inside a batch of B rows: expert << 16 | first row
  int32_t* misc;    // rows, chosen experts, segments, (spare)
  int32_t* bseg;    // [R + 1] first segment of each batch
};

__host__ __device__ inline uint32_t layer_table_bytes(int E, int R) {
  return uint32_t((4 * (3 * E + 5 * R + 4 + R + 1) + 15) & ~15);
}

__device__ __forceinline__ LayerTables layer_tables(uint8_t* p, int E, int R) {
  LayerTables t;
  int32_t* q = reinterpret_cast<int32_t*>(p);
  t.mask = q; q += E;
  t.start = q; q += E;
  t.touch = q; q += E;
  t.id = q; q += R;
  t.w = reinterpret_cast<float*>(q); q += R;
  t.row = q; q += R;
  t.roww = reinterpret_cast<float*>(q); q += R;
  t.seg = q; q += R;
  t.misc = q; q += 4;
  t.bseg = q;
  return t;
}

// Every thread of the workgroup calls it; `scratch`: E floats per wave.
template <int KPL>
__device__ __forceinline__ void build_tables(const LayerArgs& a, const LayerTables& T, float* scratch, int B) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.rt.E, topk = a.rt.topk, M = a.M, R = M * topk;
  for (int e = tid; e < E; e += kLyThreads) T.mask[e] = 0;
  __syncthreads();
  for (int t = wave; t < M; t += kLyWaves) {
    float l[KPL], b[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int e = lane * KPL + i;
      l[i] = -__builtin_huge_valf();
      b[i] = 0.f;
      if (e < E) {
        float s = a.gate_bias ? a.gate_bias[e] : 0.f;
        const float* p = a.part + int64_t(t + a.t0) * E + e;
        for (int c = 0; c < a.S; ++c) s += p[int64_t(c) * a.M_all * E];
        l[i] = s;
        if (a.rt.bias) b[i] = a.rt.bias[e];
      }
    }
    bool close;
    const RouteSlot s = route_token<KPL, float>(l, b, a.rt, scratch + wave * E, close);
    if (lane < topk) {
      T.id[t * topk + lane] = s.id;
      T.w[t * topk + lane] = s.w;
      if (s.id >= 0) atomicOr(&T.mask[s.id], 1 << t);
    }
  }
  __syncthreads();
  if (wave == 0) {
    // lane l owns a run of experts; one wave-wide scan of (rows, chosen experts)
    const int per = (E + 63) / 64;
    const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
    int nr = 0, nt = 0;
    for (int e = e0; e < e1; ++e) {
      const int c = __popc(T.mask[e]);
      nr += c;
      nt += c > 0 ? 1 : 0;
    }
    int sr = nr, sn = nt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int tr = __shfl_up(sr, o, 64), tn = __shfl_up(sn, o, 64);
      if (lane >= o) {
        sr += tr;
        sn += tn;
      }
    }
    int rb = sr - nr, tb = sn - nt;
    for (int e = e0; e < e1; ++e) {
      const int c = __popc(T.mask[e]);
      T.start[e] = rb;
      rb += c;
      if (c > 0) T.touch[tb++] = e;
    }
    if (lane == 63) {
      T.misc[0] = sr;
      T.misc[1] = sn;
    }
  }
  __syncthreads();
  for (int r = tid; r < R; r += kLyThreads) {
    const int e = T.id[r], t = r / topk;
    if (e < 0) continue;
    const int j = T.start[e] + __popc(T.mask[e] & ((1 << t) - 1));
    T.row[j] = e << 8 | t;
    T.roww[j] = T.w[r];
  }
  __syncthreads();
  if (B > 0 && wave == 0) {
    const int rows = T.misc[0];
    int n = 0;
    for (int j0 = 0; j0 < rows; j0 += 64) {
      const int j = j0 + lane;
      const bool first = j < rows && (j % B == 0 || (T.row[j] >> 8) != (T.row[j - 1] >> 8));
      const uint64_t m = __ballot(first);
      const int at = n + __popcll(m & ((uint64_t(1) << lane) - 1));
      if (first) {
        T.seg[at] = (T.row[j] >> 8) << 16 | j;
        if (j % B == 0) T.bseg[j / B] = at;
      }
      n += __popcll(m);
    }
    if (lane == 0) {
      T.misc[2] = n;
      T.bseg[(rows + B - 1) / B] = n;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- weight streams

// One 128-byte step of a lane's weight rows in the ring: G 16-row groups, lane (l16, q) holds bytes
// [32 q, +32) of row l16's step (the same bytes from both layouts), with what scales them: MXFP4
// the two e8m0 codes of those bytes' 32-element groups; FP8 the 128 x 128 block's scale.
template <int WFMT, int G>
struct WStep {
  i32x4 w[G][2];
  uint32_t s[G][WFMT == W_E2M1_MX ? 2 : 1];
};

// Where a 16-row group's bytes come from.
template <int G>
struct WGeo {
  const uint8_t* w;   // expert base (uniform)
  const uint8_t* s;
  uint32_t woff[G];   // plain: row * row_bytes;  tiled: first tile of the group + 16 lane
  uint32_t soff[G];   // MXFP4 plain: row * groups, tiled: first tile + 2 lane;  FP8: byte offset of the block row
};

// Matrix of one stage: [E][N rows][K].
struct WMat {
  const uint8_t* w;
  const uint8_t* s;
  int64_t w_estride, s_estride;  // bytes per expert
  int32_t N, K, nsteps;
};

template <int WFMT>
__device__ __forceinline__ constexpr int wstep_elems() { return WFMT == W_E2M1_MX ? 256 : 128; }

template <int WFMT, bool TILED>
__device__ __forceinline__ WMat wmat(const uint8_t* w, const uint8_t* s, int N, int K) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  WMat m;
  m.w = w;
  m.s = s;
  m.N = N;
  m.K = K;
  m.nsteps = (K + wstep_elems<WFMT>() - 1) / wstep_elems<WFMT>();
  const int64_t row = MX ? K / 2 : K;
  m.w_estride = int64_t(N) * (TILED ? int64_t(m.nsteps) * 128 : row);
  m.s_estride = MX ? int64_t(N) * (TILED ? m.nsteps * 8 : K / 32) : int64_t((N + 127) / 128) * (K / 128) * 4;
  return m;
}

// Geometry of group g of expert e: rows [16 grp, +16).
template <int WFMT, bool TILED, int G>
__device__ __forceinline__ void geo_group(WGeo<G>& o, const WMat& m, int g, int grp) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  if (TILED) {
    o.woff[g] = uint32_t(grp) * uint32_t(m.nsteps) * 2048u + uint32_t(lane) * 16u;
    if (MX) o.soff[g] = uint32_t(grp) * uint32_t(m.nsteps) * 128u + uint32_t(lane) * 2u;
  } else {
    const uint32_t row = uint32_t(grp) * 16u + uint32_t(l16);
    o.woff[g] = row * uint32_t(MX ? m.K / 2 : m.K);
    if (MX) o.soff[g] = row * uint32_t(m.K / 32);
  }
  if (!MX) o.soff[g] = uint32_t(grp >> 3) * uint32_t(m.K / 128) * 4u;
}

// `vzero`: a zero the compiler does not know to be one, in a vector register, so that the FP8 block
// scales come through the vector memory path like the weights (a scalar load would share its
// counter with the LDS reads, which would then wait for it).
template <int WFMT, bool TILED, int G>
__device__ __forceinline__ void wload(WStep<WFMT, G>& o, const WGeo<G>& gm, const WMat& m, int st, uint32_t vzero) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const uint32_t sc = uint32_t(st);
  if constexpr (TILED) {
    // a row that ends inside its last step is zero-padded there; its padding chunks re-read the
    // row's first chunk of that step (a line lanes 0-15 fetch anyway)
    uint32_t h0 = 0u, h1 = 1024u;
    if (MX && st == m.nsteps - 1) {
      const uint32_t rest = uint32_t(m.K / 2 - (m.nsteps - 1) * 128);
      if (32u * uint32_t(q) + 16u > rest) h0 = 0u - 256u * uint32_t(q);
      if (32u * uint32_t(q) + 32u > rest) h1 = 0u - 256u * uint32_t(q);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      o.w[g][0] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(gm.w + (gm.woff[g] + sc * 2048u + h0)));
      o.w[g][1] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(gm.w + (gm.woff[g] + sc * 2048u + h1)));
      if (MX) {
        const uint32_t v = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(gm.s + gm.soff[g] + sc * 128u));
        o.s[g][0] = v;
      }
    }
  } else {
    const uint32_t row_bytes = uint32_t(MX ? m.K / 2 : m.K);
    uint32_t b0 = sc * 128u + uint32_t(q) * 32u, b1 = b0 + 16u;
    const uint32_t ngroups = uint32_t(m.K / 32);
    const uint32_t g0 = min(sc * 8u + 2u * uint32_t(q), ngroups - 1), g1 = min(sc * 8u + 2u * uint32_t(q) + 1u, ngroups - 1);
    // 16-byte chunks past the row's end re-read its first one: finite codes times zero padding
    if (MX && b0 >= row_bytes) b0 = 0;
    if (MX && b1 >= row_bytes) b1 = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      o.w[g][0] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(gm.w + (gm.woff[g] + b0)));
      o.w[g][1] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(gm.w + (gm.woff[g] + b1)));
      if constexpr (MX) {
        o.s[g][0] = gm.s[gm.soff[g] + g0];
        o.s[g][1] = gm.s[gm.soff[g] + g1];
      }
    }
  }
  if constexpr (!MX) {
#pragma unroll
    for (int g = 0; g < G; ++g)
      o.s[g][0] = *reinterpret_cast<const uint32_t*>(gm.s + (gm.soff[g] + sc * 4u + vzero));
  }
}

// acc[g] += A-step x weight-step.  arow: this lane's LDS row (its 16-byte-aligned start).
template <int WFMT, bool TILED, int G>
__device__ __forceinline__ void wcompute(f32x4 (&acc)[G], const WStep<WFMT, G>& v, const uint8_t* arow, int st) {
  const int lane = threadIdx.x & 63, q = lane >> 4;
  if constexpr (WFMT == W_E2M1_MX) {
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const i32x4 af = *reinterpret_cast<const i32x4*>(arow + (st * 256 + q * 64 + 8 * s) * 2);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t o[4];
        const uint32_t e = TILED ? (v.s[g][0] >> (8 * (s >> 2))) & 0xffu : v.s[g][s >> 2];
        e2m1x8_to_bf16(uint32_t(v.w[g][s >> 2][s & 3]), e8m0_to_f32(e), o);
        acc[g] = mfma_16x16x32_bf16(af, i32x4{int(o[0]), int(o[1]), int(o[2]), int(o[3])}, acc[g]);
      }
    }
  } else {
    f32x4 part[G];
#pragma unroll
    for (int g = 0; g < G; ++g) part[g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const i32x4 af = *reinterpret_cast<const i32x4*>(arow + (st * 128 + q * 32 + 8 * s) * 2);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t o0, o1, o2, o3;
        e4m3x4_to_bf16(uint32_t(v.w[g][s >> 1][(2 * s) & 3]), o0, o1);
        e4m3x4_to_bf16(uint32_t(v.w[g][s >> 1][(2 * s + 1) & 3]), o2, o3);
        part[g] = mfma_16x16x32_bf16(af, i32x4{int(o0), int(o1), int(o2), int(o3)}, part[g]);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float s = __uint_as_float(v.s[g][0]);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[g][r] = fmaf(part[g][r], s, acc[g][r]);
    }
  }
}

__device__ __forceinline__ uint32_t opaque_zero() {
  uint32_t z;
  asm volatile("v_mov_b32 %0, 0" : "=v"(z));
  return z;
}

// ---------------------------------------------------------------- gate / up

// LDS: tables | x rows [M][row_stride] (the routing's group scratch lies there first)
__host__ __device__ inline uint32_t layer_row_stride(bool mx, int K) {
  const int st = mx ? 256 : 128;
  return uint32_t((K + st - 1) / st * st * 2 + 16);  // +16 B: rows read together fall in different banks
}

template <int WFMT, bool TILED, int KPL>
__global__ __launch_bounds__(kLyThreads, 2) void moe_up_kernel(LayerArgs a) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  constexpr int D = kUpD;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int E = a.rt.E, R = a.M * a.rt.topk, H = int(a.H), I = int(a.I);
  const LayerTables T = layer_tables(smem, E, R);
  uint8_t* const xs = smem + layer_table_bytes(E, R);
  build_tables<KPL>(a, T, reinterpret_cast<float*>(xs), 0);

  // ---- the tokens' rows into LDS, zero-padded to whole steps
  const uint32_t stride = layer_row_stride(MX, H);
  const int chunks = int(stride / 16) - 1, valid = H / 8;
  for (int c = tid; c < a.M * chunks; c += kLyThreads) {
    const int t = c / chunks, cc = c - t * chunks;
    i32x4 v = {0, 0, 0, 0};
    if (cc < valid) v = *reinterpret_cast<const i32x4*>(a.x + (t + a.t0) * a.ldx + cc * 8);
    *reinterpret_cast<i32x4*>(xs + t * stride + cc * 16) = v;
  }
  __syncthreads();

  // ---- items: (chosen expert, 16 gate + 16 up columns), dealt over the workgroups first
  const WMat m = wmat<WFMT, TILED>(a.w1, a.s1, 2 * I, H);
  const int tiles = I / 16, total = T.misc[1] * tiles;
  const int step = int(gridDim.x) * kLyWaves;
  int item = wave * int(gridDim.x) + int(blockIdx.x);
  if (item >= total) return;
  const uint32_t vz = opaque_zero();
  auto geo_of = [&](int it) __attribute__((always_inline)) {
    WGeo<2> g;
    const int ti = it / tiles, nt = it - ti * tiles;
    const int e = __builtin_amdgcn_readfirstlane(T.touch[ti]);
    g.w = m.w + int64_t(e) * m.w_estride;
    g.s = m.s + int64_t(e) * m.s_estride;
    geo_group<WFMT, TILED, 2>(g, m, 0, nt);
    geo_group<WFMT, TILED, 2>(g, m, 1, tiles + nt);
    return g;
  };
  WStep<WFMT, 2> ring[D];
  // load cursor: runs D - 1 steps ahead of the computation, into the next items; past the last
  // one it stays on the last step (read again, never computed)
  int lit = item, lst = 0;
  WGeo<2> lg = geo_of(lit);
  auto load = [&](int slot) __attribute__((always_inline)) {
    wload<WFMT, TILED, 2>(ring[slot], lg, m, lst, vz);
    if (lst + 1 < m.nsteps) {
      ++lst;
    } else if (lit + step < total) {
      lit += step;
      lst = 0;
      lg = geo_of(lit);
    }
  };
#pragma unroll
  for (int u = 0; u < D - 1; ++u) load(u);

  f32x4 acc[2];
  const uint8_t* arow = xs;
  int rows = 0, row0 = 0, st = 0, nt = 0, ex = 0;
  float bg = 0.f, bu = 0.f;
  auto begin = [&]() __attribute__((always_inline)) {
    const int ti = item / tiles;
    nt = item - ti * tiles;
    ex = __builtin_amdgcn_readfirstlane(T.touch[ti]);
    rows = __builtin_amdgcn_readfirstlane(__popc(T.mask[ex]));
    row0 = __builtin_amdgcn_readfirstlane(T.start[ex]);
    arow = xs + uint32_t(T.row[row0 + min(l16, rows - 1)] & 0xff) * stride;
    acc[0] = acc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    st = 0;
    // (read here, behind the ring's requests so far: in finish() the wait for it would drain the ring)
    if (a.b1) {
      const float* be = a.b1 + int64_t(ex) * 2 * I + nt * 16 + l16;
      bg = be[0];
      bu = be[I];
    }
  };
  auto finish = [&]() __attribute__((always_inline)) {
    const int col = nt * 16 + l16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 4 * q + r;
      if (i >= rows) continue;
      const float g = acc[0][r] + bg, u = acc[1][r] + bu;
      const float h = T.roww[row0 + i] * (g / (1.0f + __expf(-g)) * u);
      const uint16_t hi = f2bf(h);
      const float hf = bf16f(hi);
      const uint16_t lo = f2bf(fabsf(hf) < __builtin_huge_valf() ? h - hf : 0.f);
      uint16_t* o = a.h + int64_t(row0 + i) * 2 * I + col;
      o[0] = hi;
      o[I] = lo;
    }
  };
  begin();
  for (bool more = true; more;) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      load((u + D - 1) % D);
      if (more) {
        wcompute<WFMT, TILED, 2>(acc, ring[u], arow, st);
        if (++st == m.nsteps) {
          finish();
          item += step;
          more = item < total;
          if (more) begin();
        }
      }
    }
  }
}

// ---------------------------------------------------------------- down

__host__ __device__ inline uint32_t layer_down_part_bytes(int B) { return uint32_t(2 * kLyWaves * B * 16 * 4); }

// LDS: tables | partial sums [2][8 waves][B][16] fp32 | h rows [nbuf][B][hi, lo][row_stride]
template <int WFMT, bool TILED, int KPL>
__global__ __launch_bounds__(kLyThreads, 2) void moe_down_kernel(LayerArgs a) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  constexpr int D = kDownD;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int E = a.rt.E, R = a.M * a.rt.topk, H = int(a.H), I = int(a.I), B = a.B;
  const LayerTables T = layer_tables(smem, E, R);
  float* const part = reinterpret_cast<float*>(smem + layer_table_bytes(E, R));
  const uint32_t hs_off = layer_table_bytes(E, R) + layer_down_part_bytes(B);
  uint8_t* const hs = smem + hs_off;
  const uint32_t hs_addr = lds_addr(smem) + hs_off;
  build_tables<KPL>(a, T, reinterpret_cast<float*>(hs), B);

  const uint32_t stride = layer_row_stride(MX, I), buf_bytes = uint32_t(2 * B) * stride;
  const int rows = __builtin_amdgcn_readfirstlane(T.misc[0]);
  const int nb = (rows + B - 1) / B;  // batches per item
  const WMat m = wmat<WFMT, TILED>(a.w2, a.s2, H, I);
  const int items = H / 16;
  const int my = items > int(blockIdx.x) ? (items - 1 - int(blockIdx.x)) / int(gridDim.x) + 1 : 0;

  // tokens with no expert at all, or none anywhere
  const int tok = tid >> 4, tc = tid & 15;
  if (nb == 0) {
    for (int i = 0; i < my; ++i)
      if (tok < a.M) a.out[(tok + a.t0) * a.ldo + (int64_t(blockIdx.x) + int64_t(i) * gridDim.x) * 16 + tc] = 0;
    return;
  }
  if (my == 0) return;

  // zero the rows' padding to whole steps (the copies below write [0, I) of a row), and the sums
  {
    const int pad = int(stride / 16) - I / 8;
    const int nrow = 2 * B * (nb > 1 ? 2 : 1);
    for (int c = tid; c < nrow * pad; c += kLyThreads)
      *reinterpret_cast<i32x4*>(hs + uint32_t(c / pad) * stride + uint32_t(I / 8 + c % pad) * 16) = i32x4{0, 0, 0, 0};
    for (int c = tid; c < 2 * kLyWaves * B * 16; c += kLyThreads) part[c] = 0.f;
  }

  // rows of batch b (I bf16 hi, then I lo, one after the other in memory) into LDS buffer `buf`
  const int segs = (I * 2 + 1023) / 1024;
  auto copy_batch = [&](int b, int buf) __attribute__((always_inline)) {
    const int j0 = b * B, n = min(B, rows - j0) * 2;
    for (int i = wave; i < n * segs; i += kLyWaves) {
      const int r = i / segs, s = i - r * segs;
      const int64_t cb = int64_t(s) * 1024 + lane * 16;
      if (cb < I * 2)
        lds_dma16(reinterpret_cast<const uint8_t*>(a.h) + (int64_t(j0) * 2 + r) * I * 2 + cb,
                  hs_addr + uint32_t(buf) * buf_bytes + uint32_t(r) * stride + uint32_t(s) * 1024u);
    }
  };

  // this wave's share of batch b: steps [lo, hi) of its segments' nsteps each
  struct Share { int seg0, lo, hi; };
  auto share = [&](int b) __attribute__((always_inline)) {
    Share s;
    s.seg0 = __builtin_amdgcn_readfirstlane(T.bseg[b]);
    const int n = (__builtin_amdgcn_readfirstlane(T.bseg[b + 1]) - s.seg0) * m.nsteps;
    s.lo = n * wave / kLyWaves;
    s.hi = n * (wave + 1) / kLyWaves;
    return s;
  };
  const uint32_t vz = opaque_zero();
  const int nv = my * nb;  // (item, batch) pairs
  auto geo_of = [&](int v, int seg) __attribute__((always_inline)) {
    WGeo<1> g;
    const int e = __builtin_amdgcn_readfirstlane(T.seg[seg]) >> 16;
    g.w = m.w + int64_t(e) * m.w_estride;
    g.s = m.s + int64_t(e) * m.s_estride;
    geo_group<WFMT, TILED, 1>(g, m, 0, int(blockIdx.x) + (v / nb) * int(gridDim.x));
    return g;
  };

  // load cursor: pair lv, its share's step lp (of lhi), as segment lseg, step lst
  int lv = -1, lp = 0, lhi = 0, lseg = 0, lst = 0;
  WGeo<1> lg{};
  auto next_pair = [&]() __attribute__((always_inline)) {  // the next pair with work for this wave, if any
    int v = lv + 1;
    while (v < nv) {
      const Share s = share(v % nb);
      if (s.hi > s.lo) {
        lv = v;
        lp = s.lo;
        lhi = s.hi;
        lseg = s.seg0 + s.lo / m.nsteps;
        lst = s.lo % m.nsteps;
        lg = geo_of(v, lseg);
        return;
      }
      ++v;
    }
  };
  next_pair();
  const bool any = lv >= 0;  // (a wave may have no work at all: it only joins the barriers)
  if (!any) {
    lg = geo_of(0, 0);
  }
  WStep<WFMT, 1> ring[D];
  int issued = 0;  // ring steps requested since the last batch copy
  auto load = [&](int slot) __attribute__((always_inline)) {
    wload<WFMT, TILED, 1>(ring[slot], lg, m, lst, vz);
    ++issued;
    if (lp + 1 < lhi) {
      ++lp;
      if (++lst == m.nsteps) {
        lst = 0;
        ++lseg;
        lg = geo_of(lv, lseg);
      }
    } else {
      next_pair();  // past the last pair: the cursor stays (its last step is read again, never computed)
    }
  };

  __syncthreads();  // the zeroed padding, before the copies
  copy_batch(0, 0);
#pragma unroll
  for (int u = 0; u < D - 1; ++u) load(u);

  f32x4 acc[1];
  const uint8_t* arow = hs;
  float sum = 0.f;  // out[tok][tc] of the current item (threads below 256)
  int v = 0, b = 0, cp = 0, chi = 0, cseg = 0, cst = 0, j0 = 0, sm = 0;

  auto begin_seg = [&]() __attribute__((always_inline)) {
    const int sg = __builtin_amdgcn_readfirstlane(T.seg[cseg]);
    j0 = sg & 0xffff;
    const int end = cseg + 1 < __builtin_amdgcn_readfirstlane(T.bseg[b + 1])
                        ? (__builtin_amdgcn_readfirstlane(T.seg[cseg + 1]) & 0xffff) : min(rows, (b + 1) * B);
    sm = end - j0;
    const int i = l16 & 7;
    arow = hs + uint32_t(nb > 1 ? (v & 1) : 0) * buf_bytes +
           uint32_t(2 * (j0 - b * B + (i < sm ? i : 0)) + (l16 >> 3)) * stride;
    acc[0] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  // MFMA rows i and i + 8 are the two terms of h row i
  auto end_seg = [&]() __attribute__((always_inline)) {
    f32x4 o;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = acc[0][r] + __shfl_xor(acc[0][r], 32, kWave);
    float* p = part + ((v & 1) * kLyWaves + wave) * B * 16 + (j0 - b * B) * 16 + l16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 4 * q + r;
      if (q < 2 && i < sm) p[i * 16] = o[r];
    }
  };
  auto begin_pair = [&]() __attribute__((always_inline)) {
    const Share s = share(b);
    cp = s.lo;
    chi = s.hi;
    cseg = s.seg0 + s.lo / m.nsteps;
    cst = s.lo % m.nsteps;
    if (cp < chi) begin_seg();
  };
  // pair v is done: publish its sums, take over the next batch's rows, add up pair v's sums
  auto end_pair = [&]() __attribute__((always_inline)) {
    const bool last_batch = b == nb - 1;
    if (nb > 1 && v + 1 < nv) {
      // the copies of pair v + 1's rows were issued before `issued` ring steps, each of at least
      // two reads
      if (issued >= D - 1)
        wait_vmcnt<(D - 1) * 2>();
      else
        wait_vmcnt<0>();
    }
    __syncthreads();
    if (nb > 1 && v + 2 < nv) {
      copy_batch((v + 2) % nb, v & 1);
      issued = 0;
    }
    if (tid < 256) {
      const float* p = part + (v & 1) * kLyWaves * B * 16;
      const int n = min(B, rows - b * B);
      for (int i = 0; i < n; ++i) {
        if ((T.row[b * B + i] & 0xff) != tok) continue;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kLyWaves; ++w) s += p[(w * B + i) * 16 + tc];
        sum += s;
      }
      if (last_batch) {
        if (tok < a.M)
          a.out[(tok + a.t0) * a.ldo + (int64_t(blockIdx.x) + int64_t(v / nb) * gridDim.x) * 16 + tc] = f2bf(sum);
        sum = 0.f;
      }
    }
    __syncthreads();
    // clear this wave's sums for pair v + 2
    for (int c = lane; c < B * 16; c += 64) part[((v & 1) * kLyWaves + wave) * B * 16 + c] = 0.f;
    ++v;
    b = last_batch ? 0 : b + 1;
  };

  wait_vmcnt<0>();
  __syncthreads();
  if (nb > 1 && nv > 1) {
    copy_batch(1 % nb, 1);
    issued = 0;
  }
  begin_pair();
  while (v < nv) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      load((u + D - 1) % D);
      while (v < nv && cp >= chi) {  // also pairs without work for this wave
        end_pair();
        if (v < nv) begin_pair();
      }
      if (v < nv) {
        wcompute<WFMT, TILED, 1>(acc, ring[u], arow, cst);
        ++cp;
        if (++cst == m.nsteps || cp == chi) {
          end_seg();
          cst = 0;
          ++cseg;
          if (cp < chi) begin_seg();
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host side

namespace {
constexpr uint32_t kLyMaxLds = 156 * 1024;  // of 160 KB

int layer_cus() {
  static int cus[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (cus[dev] <= 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    cus[dev] = n;
  }
  return cus[dev];
}

// the larger of the stage's operands and the routing's group scratch (E floats per wave)
uint32_t with_scratch(uint32_t bytes, int E) { return std::max(bytes, uint32_t(kLyWaves * E * 4)); }

uint32_t up_lds(bool mx, int64_t H, int E, int topk, int M) {
  return layer_table_bytes(E, M * topk) + with_scratch(uint32_t(M) * layer_row_stride(mx, int(H)), E);
}

uint32_t down_lds(bool mx, int64_t I, int E, int rows, int B) {
  return layer_table_bytes(E, rows) + layer_down_part_bytes(B) +
         with_scratch(uint32_t((rows > B ? 2 : 1) * 2 * B) * layer_row_stride(mx, int(I)), E);
}

template <int WFMT, bool TILED, int KPL>
void launch_layer_t(const LayerArgs& a, hipStream_t st) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  const int R = a.M * a.rt.topk;
  const int64_t most = std::min<int64_t>(a.rt.E, R);  // chosen experts at most
  const unsigned gu = unsigned(std::min<int64_t>(layer_cus(), cdiv(most * (a.I / 16), kLyWaves)));
  hipLaunchKernelGGL((moe_up_kernel<WFMT, TILED, KPL>), dim3(gu), dim3(kLyThreads),
                     up_lds(MX, a.H, a.rt.E, a.rt.topk, a.M), st, a);
  const unsigned gd = unsigned(std::min<int64_t>(layer_cus(), a.H / 16));
  hipLaunchKernelGGL((moe_down_kernel<WFMT, TILED, KPL>), dim3(gd), dim3(kLyThreads),
                     down_lds(MX, a.I, a.rt.E, R, a.B), st, a);
}

template <int WFMT, bool TILED>
void launch_layer_k(const LayerArgs& a, hipStream_t st) {
  if (a.rt.E <= 128) launch_layer_t<WFMT, TILED, 2>(a, st);
  else if (a.rt.E <= 256) launch_layer_t<WFMT, TILED, 4>(a, st);
  else launch_layer_t<WFMT, TILED, 8>(a, st);
}
}  // namespace

int layer_pass_tokens(int wfmt, int64_t H, int32_t E, int32_t topk) {
  int m = kLayerMaxTokens;
  while (m > 0 && up_lds(wfmt == W_E2M1_MX, H, E, topk, m) > kLyMaxLds) --m;
  return m;
}

int layer_batch_rows(int wfmt, int64_t I, int32_t E, int32_t rows) {
  int B = 8;
  while (B > 0 && down_lds(wfmt == W_E2M1_MX, I, E, rows, B) > kLyMaxLds) B /= 2;
  return B;
}

// Enough workgroups to read the router's weights from all over the GPU, chunks of at least 512.
void layer_gate_split(int32_t E, int64_t H, int32_t& S, int32_t& chunk) {
  const int64_t tiles = cdiv(E, 16);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>({cdiv(256, tiles), cdiv(H, 512), 16}));
  chunk = int32_t(cdiv(cdiv(H, want), 128) * 128);
  S = int32_t(cdiv(H, chunk));
}

void launch_moe_layer(const LayerArgs& g, hipStream_t st) {
  LayerArgs a = g;
  const dim3 grid(unsigned(cdiv(a.rt.E, 16)), unsigned(a.S));
  if (a.gate_f32)
    hipLaunchKernelGGL((moe_gate_kernel<true>), grid, dim3(kGateThreads), 0, st, a.x, a.M_all, a.ldx, a.gate, a.rt.E,
                       a.H, a.chunk, a.part);
  else
    hipLaunchKernelGGL((moe_gate_kernel<false>), grid, dim3(kGateThreads), 0, st, a.x, a.M_all, a.ldx, a.gate, a.rt.E,
                       a.H, a.chunk, a.part);
  const int pass = layer_pass_tokens(a.wfmt, a.H, a.rt.E, a.rt.topk);
  for (a.t0 = 0; a.t0 < a.M_all; a.t0 += pass) {
    a.M = std::min(pass, a.M_all - a.t0);
    a.B = layer_batch_rows(a.wfmt, a.I, a.rt.E, a.M * a.rt.topk);
    if (a.wfmt == W_E2M1_MX) {
      if (a.tiled) launch_layer_k<W_E2M1_MX, true>(a, st);
      else launch_layer_k<W_E2M1_MX, false>(a, st);
    } else {
      if (a.tiled) launch_layer_k<W_E4M3_BLOCK, true>(a, st);
      else launch_layer_k<W_E4M3_BLOCK, false>(a, st);
    }
  }
}

}  // namespace mxq
