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
// weight streams: every wave requests its 128-byte row steps D - 1 ahead into registers (a ring of D), on
// across its work items, and the activations come from LDS.  In the down stage the ring stays in flight
// as written.  In gate/up the compiled waits cut it short: MXFP4's scale codes are read in 8 or 16 bits and
// widened at the end of each turn of D steps, where the wave waits for every request; FP8's first step
// of a turn waits until 8 requests of 12 are left; and a w1_bias is waited for at an item's end, behind
// the ring's requests.  Plain weights reach 3.5 to 4 TB/s there, against 5.8 in a bare read loop.
//
//  * moe_gate_kernel: the router product on V_MFMA_F32_16X16X32_BF16, split over experts and K;
//    fp32 router weights are split into three bf16 terms that sum to them exactly.  Partial sums
//    go to the workspace and are added in order where they are read.
//  * moe_up_kernel: every workgroup routes all tokens itself (one wave per token: the logits are
//    a few KB) and builds the same tables in LDS: chosen experts ascending, each with its rows
//    (tokens ascending).  An item is 16 gate columns and the 16 matching up columns of one expert;
//    a wave takes it over the whole K; where tokens agree on few experts and items are at most a quarter
//    of the waves, four or eight waves share an item's K steps and meet in LDS.
//  * moe_down_kernel: a workgroup's item is 16 output columns over ALL chosen experts; its eight
//    waves split the (segments of at most kDownRows rows of an expert) x (K steps) evenly, each
//    fetching the h rows of its own steps through registers into a few KB of LDS of its own, and
//    their sums meet in LDS once an item, each token's rows added in a fixed order -- no partial
//    outputs in memory, no atomics, no combine launch.  (A first version staged the h rows for the
//    whole workgroup, a barrier per four rows: 110 us against 60 us for 16 MXFP4 tokens.)
//
// Rounding: products and sums are fp32.  The routing weight joins h in fp32.  h is kept as two
// bf16 terms (hi + lo, relative error 2^-17 of it): with one bf16 term the output's error against
// 64 bits would be 1.4 times its own rounding.  The 16 rows of the MFMA are mostly empty here, so
// hi and lo are simply two rows of the same product.
#include <algorithm>

#include "layer.hpp"
#include "route_common.hpp"

namespace mxq {

namespace {
constexpr int kLyThreads = 512, kLyWaves = 8;
constexpr int kGateThreads = 256;
constexpr int kDownRows = 4;  // rows of an expert that one pass over its weights takes in the down stage
// Steps in the weight rings (that many less one requested ahead).  Depths 3 / 4, 4 / 6, 8 / 6 of gate-up /
// down took 35, 36, 41 us (one MXFP4 token) and 147, 147, 152 us (16 tokens); gate/up's turns all ended in
// a wait for every request, so this compares no deeper ring that stays in flight.
constexpr int kUpD = 3, kDownD = 4;
}  // namespace

// ---------------------------------------------------------------- router product

// Two bf16 with infinities and NaNs replaced by zeros.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v) {
  const uint32_t lo = (v & 0x7f80u) == 0x7f80u ? 0u : 0xffffu, hi = (v & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u;
  return v & (lo | hi);
}

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
      const float v0[8] = {g0[0], g0[1], g0[2], g0[3], g1[0], g1[1], g1[2], g1[3]};
      float v[8] = {g0[0], g0[1], g0[2], g0[3], g1[0], g1[1], g1[2], g1[3]};
      // v = t0 + t1 + t2 with bf16 terms: each term cuts off the next eight bits of the significand (cut, not
      // rounded: a weight above bf16's largest finite value would round to infinity).  An infinite
      // activation meets only the first, which has v's sign: the others may be zero.
      i32x4 fin;
#pragma unroll
      for (int i = 0; i < 4; ++i) fin[i] = int(finite_bf16x2(uint32_t(af[i])));
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        i32x4 b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t lo = __float_as_uint(v[2 * i]) & 0xffff0000u, hi = __float_as_uint(v[2 * i + 1]) & 0xffff0000u;
          v[2 * i] -= __uint_as_float(lo);
          v[2 * i + 1] -= __uint_as_float(hi);
          if (term == 0) {
            // an infinite or NaN weight stays what it is and has no remainder
            const uint32_t w = pack_bf16x2(v0[2 * i], v0[2 * i + 1]);
            if (!(fabsf(v0[2 * i]) < __builtin_huge_valf())) {
              lo = w << 16;
              v[2 * i] = 0.f;
            }
            if (!(fabsf(v0[2 * i + 1]) < __builtin_huge_valf())) {
              hi = w & 0xffff0000u;
              v[2 * i + 1] = 0.f;
            }
          }
          b[i] = int(hi | lo >> 16);
        }
        acc = mfma_16x16x32_bf16(term == 0 ? af : fin, b, acc);
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

// What the gate/up stage needs to know about the routing.
struct UpTables {
  int32_t* mask;    // [E] tokens of each expert, one bit per token
  int32_t* start;   // [E] first sorted row of each expert
  int32_t* touch;   // [E] chosen experts, ascending
  int32_t* id;      // [R] expert of flat row t * topk + k
  float* w;         // [R]
  int32_t* row;     // [R] sorted rows: expert << 8 | token
  float* roww;      // [R] their routing weights
  int32_t* misc;    // rows, chosen experts
};

__host__ __device__ inline uint32_t up_table_bytes(int E, int R) { return uint32_t((4 * (3 * E + 4 * R + 2) + 15) & ~15); }

__device__ __forceinline__ UpTables up_tables(uint8_t* p, int E, int R) {
  UpTables t;
  int32_t* q = reinterpret_cast<int32_t*>(p);
  t.mask = q; q += E;
  t.start = q; q += E;
  t.touch = q; q += E;
  t.id = q; q += R;
  t.w = reinterpret_cast<float*>(q); q += R;
  t.row = q; q += R;
  t.roww = reinterpret_cast<float*>(q); q += R;
  t.misc = q;
  return t;
}

// Routes the pass's tokens and groups their rows by expert.  Every thread of the workgroup calls
// it; `scratch`: E doubles per wave (read where the router has groups).  As in moe_route_kernel, a token
// with picks too close for fp32 scores is routed again in 64 bits, on the same fp32 logits.
template <int KPL>
__device__ __forceinline__ void build_tables(const LayerArgs& a, const UpTables& T, double* scratch) {
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
        l[i] = a.gate_bias ? a.gate_bias[e] : 0.f;
        if (a.rt.bias) b[i] = a.rt.bias[e];
      }
    }
    // the K chunks' sums in chunk order, four chunks' reads on their way together
    const float* p = a.part + int64_t(t + a.t0) * E + lane * KPL;
    const int64_t slice = int64_t(a.M_all) * E;
    for (int c0 = 0; c0 < a.S; c0 += 4) {
      float v[4][KPL];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < KPL; ++i)
          v[c][i] = lane * KPL + i < E && c0 + c < a.S ? p[(c0 + c) * slice + i] : 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < KPL; ++i) l[i] += v[c][i];
    }
    bool close;
    RouteSlot s = route_token<KPL, float>(l, b, a.rt, reinterpret_cast<float*>(scratch + wave * E), close);
    if (__builtin_expect(close, 0)) {  // (one token's layer: 0.4 us for the repeat's code, 0.6 to 0.9 without the hint)
      bool unused;
      s = route_token<KPL, double>(l, b, a.rt, scratch + wave * E, unused);
    }
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
    const int j = e < 0 ? -1 : T.start[e] + __popc(T.mask[e] & ((1 << t) - 1));
    if (blockIdx.x == 0) a.rows[1 + R + r] = j;  // for the down stage
    if (j < 0) continue;
    T.row[j] = e << 8 | t;
    T.roww[j] = T.w[r];
  }
  __syncthreads();
}

// The down stage's: the sorted rows, and their segments -- at most kDownRows rows of one expert.
struct DownTables {
  int32_t* pos;     // [R] sorted row of flat row t * topk + k, -1: none
  int32_t* segof;   // [R] segment of each sorted row
  int32_t* seg;     // [R] expert << 16 | first row
  int32_t* misc;    // segments
};

__host__ __device__ inline uint32_t down_table_bytes(int R) { return uint32_t((4 * (3 * R + 1) + 15) & ~15); }

__device__ __forceinline__ DownTables down_tables(uint8_t* p, int R) {
  int32_t* q = reinterpret_cast<int32_t*>(p);
  return DownTables{q, q + R, q + 2 * R, q + 3 * R};
}

// ---------------------------------------------------------------- weight streams

// One 128-byte step of a lane's weight rows in the ring: G 16-row groups, lane (l16, q) holds bytes
// [64 h + 16 q, +16), h = 0, 1, of row l16's step, so one read of a wave takes whole 64-byte pieces
// of the plain layout's rows (256-byte pieces of the tiled layout) -- with half-filled pieces
// (32 q + 16 h) the plain layout's layer of one MXFP4 token took 63 us against 36 us tiled.  With
// them what scales them: MXFP4 the e8m0 codes of those bytes' 32-element groups; FP8 the 128 x 128
// block's scale.
template <int WFMT, int G>
struct WStep {
  i32x4 w[G][2];
  uint32_t s[G][WFMT == W_E2M1_MX ? 2 : 1];
};

// Where 16-row groups' bytes come from: one expert's weights and scales as buffers, this lane's
// byte offsets in them.
template <int G>
struct WGeo {
  __amdgpu_buffer_rsrc_t w, s;
  uint32_t woff[G];   // plain: row * row bytes + 16 q;  tiled: the lane's first byte in the group's first tile
  uint32_t soff[G];   // MXFP4 plain: row * groups + q, tiled: likewise;  FP8: the block row
};

// How weights lie: the plain layout; the tiled one; MXFP4's plain one with the e8m0 codes read in
// pairs, where pairs are aligned (K % 64 == 0): a lane row takes the pair that lies there and the
// codes then move between lane rows, one read of 16 rows' pieces per group and step instead of two
// (one MXFP4 token 34.6 us against 36.2, 16 tokens 207 against 212).
constexpr int kPlain = 0, kTiled = 1, kPlainPairs = 2;

// Matrix of one stage: [E][N rows][K].
struct WMat {
  const uint8_t* w;
  const uint8_t* s;
  int64_t w_estride, s_estride;  // bytes per expert
  int32_t N, K, nsteps;
};

template <int WFMT>
__device__ __forceinline__ constexpr int wstep_elems() { return WFMT == W_E2M1_MX ? 256 : 128; }

template <int WFMT, int LAY>
__device__ __forceinline__ WMat wmat(const uint8_t* w, const uint8_t* s, int N, int K) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  WMat m;
  m.w = w;
  m.s = s;
  m.N = N;
  m.K = K;
  m.nsteps = (K + wstep_elems<WFMT>() - 1) / wstep_elems<WFMT>();
  const int64_t row = MX ? K / 2 : K;
  m.w_estride = int64_t(N) * (LAY == kTiled ? int64_t(m.nsteps) * 128 : row);
  m.s_estride = MX ? int64_t(N) * (LAY == kTiled ? m.nsteps * 8 : K / 32) : int64_t((N + 127) / 128) * (K / 128) * 4;
  return m;
}

constexpr uint32_t kNoRead = 0x80000000u;  // a byte offset past every buffer's end (the host keeps them below)
constexpr int kRaw = 0x00027000;           // a raw buffer resource's last word

__device__ __forceinline__ __amdgpu_buffer_rsrc_t raw_buffer(const uint8_t* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, int(bytes), kRaw);
}

// Expert e's buffers.  Reads past a buffer's end return zeros and touch no memory.
template <int G>
__device__ __forceinline__ void geo_expert(WGeo<G>& o, const WMat& m, int e) {
  o.w = raw_buffer(m.w + int64_t(e) * m.w_estride, uint32_t(m.w_estride));
  o.s = raw_buffer(m.s + int64_t(e) * m.s_estride, uint32_t(m.s_estride));
}

// One of two geometries by a uniform choice.
template <int G>
__device__ __forceinline__ WGeo<G> geo_pick(bool second, const WGeo<G>& a, const WGeo<G>& b) {
  WGeo<G> o;
  o.w = second ? b.w : a.w;
  o.s = second ? b.s : a.s;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    o.woff[g] = second ? b.woff[g] : a.woff[g];
    o.soff[g] = second ? b.soff[g] : a.soff[g];
  }
  return o;
}

// Group g is the 16 rows [16 grp, +16).
template <int WFMT, int LAY, int G>
__device__ __forceinline__ void geo_group(WGeo<G>& o, const WMat& m, int g, int grp) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  if (LAY == kTiled) {
    // bytes 64 h + 16 q of a row's step are chunk (q & 1) of lane group 2 h + q / 2 in the tile
    o.woff[g] = uint32_t(grp) * uint32_t(m.nsteps) * 2048u + uint32_t((q & 1) * 1024 + (q >> 1) * 256 + l16 * 16);
    if (MX) o.soff[g] = uint32_t(grp) * uint32_t(m.nsteps) * 128u + uint32_t((q & 1) + (q >> 1) * 32 + l16 * 2);
  } else {
    const uint32_t row = uint32_t(grp) * 16u + uint32_t(l16);
    o.woff[g] = row * uint32_t(MX ? m.K / 2 : m.K) + uint32_t(q) * 16u;
    if (MX) o.soff[g] = row * uint32_t(m.K / 32) + uint32_t(LAY == kPlainPairs ? 2 * q : q);
  }
  if (!MX) o.soff[g] = uint32_t(grp >> 3) * uint32_t(m.K / 128) * 4u;
}

// Step st (uniform) of the groups: the lane offsets stay as they are along a row, the step goes into
// the scalar offset.  Nothing is read past st_end, nor of chunks past a row's end (MXFP4 rows that
// end inside a step).
template <int WFMT, int LAY, int G>
__device__ __forceinline__ void wload(WStep<WFMT, G>& o, const WGeo<G>& gm, const WMat& m, int st, int st_end) {
  constexpr bool MX = WFMT == W_E2M1_MX, TILED = LAY == kTiled;
  // the tiled layout's pieces are read once and whole: non-temporal (6.6 against 5.9 TB/s streaming);
  // the plain layout's 64-byte pieces want the line's other half to stay (5.1 against 5.7 TB/s)
  constexpr int kNt = TILED ? 2 : 0;
  const int q = (threadIdx.x & 63) >> 4;
  const bool dead = st >= st_end;
  // (a dead step's scalar offset could lie behind the buffer's end, of which the lanes' offsets are held
  // to be short by just that much)
  const int live = dead ? 0 : st, wo = live * (TILED ? 2048 : 128), so = MX ? live * (TILED ? 128 : 8) : live * 4;
  bool no0 = dead, no1 = dead, nop = dead;
  if (MX) {
    const int rest = m.K / 2 - (m.nsteps - 1) * 128 - q * 16;  // bytes of the last step from this lane's first
    const bool last = st == m.nsteps - 1;
    no0 = dead || (last && rest <= 0);
    no1 = dead || (last && rest <= 64);
    nop = dead || (last && m.K / 32 - (m.nsteps - 1) * 8 <= 2 * q);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint32_t w0 = no0 ? kNoRead : gm.woff[g], w1 = no1 ? kNoRead : gm.woff[g] + (TILED ? 512u : 64u);
    o.w[g][0] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(gm.w, w0, wo, kNt));
    o.w[g][1] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(gm.w, w1, wo, kNt));
    if constexpr (MX && LAY == kPlainPairs) {
      o.s[g][0] = __builtin_amdgcn_raw_buffer_load_b16(gm.s, nop ? kNoRead : gm.soff[g], so, 0);
    } else if constexpr (MX) {
      const uint32_t s0 = no0 ? kNoRead : gm.soff[g], s1 = no1 ? kNoRead : gm.soff[g] + (TILED ? 64u : 4u);
      o.s[g][0] = __builtin_amdgcn_raw_buffer_load_b8(gm.s, s0, so, 0);
      o.s[g][1] = __builtin_amdgcn_raw_buffer_load_b8(gm.s, s1, so, 0);
    } else {
      o.s[g][0] = __builtin_amdgcn_raw_buffer_load_b32(gm.s, dead ? kNoRead : gm.soff[g], so, 0);
    }
  }
}

// The two e8m0 codes of this lane's bytes of a step: its groups are q and 4 + q of the row's eight.
// In pairs, lane row q holds groups 2 q and 2 q + 1, so it takes them from rows q / 2 and 2 + q / 2.
template <int LAY>
__device__ __forceinline__ void scale_codes(const uint32_t (&s)[2], uint32_t& c0, uint32_t& c1) {
  if constexpr (LAY == kPlainPairs) {
    const int q = (threadIdx.x & 63) >> 4;
    const auto h = __builtin_amdgcn_permlane32_swap(s[0], s[0], false, false);  // rows 0 1 0 1 | 2 3 2 3
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);  // row 0 | row 1
    const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);  // row 2 | row 3
    const uint32_t sh = uint32_t(q & 1) * 8;
    c0 = ((q < 2 ? a[0] : a[1]) >> sh) & 0xffu;
    c1 = ((q < 2 ? b[0] : b[1]) >> sh) & 0xffu;
  } else {
    c0 = s[0];
    c1 = s[1];
  }
}

// acc += step of rows held in LDS with chunk c of row r in slot c ^ r, one group.  at[i]: this lane's
// chunk i (of four, MXFP4; two, FP8) in the first half of its row's step; the second half follows
// HALF bytes on.
template <int WFMT>
struct RowAt {
  static constexpr int N = WFMT == W_E2M1_MX ? 4 : 2, HALF = WFMT == W_E2M1_MX ? 256 : 128;
  const uint8_t* p[N];
};
template <int WFMT>
__device__ __forceinline__ RowAt<WFMT> row_at(const uint8_t* base, int r) {
  constexpr int N = RowAt<WFMT>::N;
  const int q = (threadIdx.x & 63) >> 4;
  RowAt<WFMT> o;
#pragma unroll
  for (int i = 0; i < N; ++i) o.p[i] = base + r * (2 * RowAt<WFMT>::HALF) + (((q * N + i) ^ r) * 16);
  return o;
}

template <int WFMT, int LAY>
__device__ __forceinline__ void wcompute_rows(f32x4& acc, const WStep<WFMT, 1>& v, const RowAt<WFMT>& at) {
  if constexpr (WFMT == W_E2M1_MX) {
    uint32_t c0, c1;
    scale_codes<LAY>(v.s[0], c0, c1);
    const float e0 = e8m0_to_f32(c0), e1 = e8m0_to_f32(c1);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const i32x4 af = *reinterpret_cast<const i32x4*>(at.p[s & 3] + (s >> 2) * RowAt<WFMT>::HALF);
      uint32_t o[4];
      e2m1x8_to_bf16(uint32_t(v.w[0][s >> 2][s & 3]), s < 4 ? e0 : e1, o);
      acc = mfma_16x16x32_bf16(af, i32x4{int(o[0]), int(o[1]), int(o[2]), int(o[3])}, acc);
    }
  } else {
    f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const i32x4 af = *reinterpret_cast<const i32x4*>(at.p[s & 1] + (s >> 1) * RowAt<WFMT>::HALF);
      uint32_t o0, o1, o2, o3;
      e4m3x4_to_bf16(uint32_t(v.w[0][s >> 1][(2 * s) & 3]), o0, o1);
      e4m3x4_to_bf16(uint32_t(v.w[0][s >> 1][(2 * s + 1) & 3]), o2, o3);
      part = mfma_16x16x32_bf16(af, i32x4{int(o0), int(o1), int(o2), int(o3)}, part);
    }
    const float s = __uint_as_float(v.s[0][0]);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = fmaf(part[k], s, acc[k]);
  }
}

// acc[g] += A-step x weight-step.  arow: this lane's LDS row (its 16-byte-aligned start).
template <int WFMT, int LAY, int G>
__device__ __forceinline__ void wcompute(f32x4 (&acc)[G], const WStep<WFMT, G>& v, const uint8_t* arow, int st) {
  const int lane = threadIdx.x & 63, q = lane >> 4;
  if constexpr (WFMT == W_E2M1_MX) {
    float e[G][2];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      uint32_t c0, c1;
      scale_codes<LAY>(v.s[g], c0, c1);
      e[g][0] = e8m0_to_f32(c0);
      e[g][1] = e8m0_to_f32(c1);
    }
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const i32x4 af = *reinterpret_cast<const i32x4*>(arow + (st * 256 + (s >> 2) * 128 + q * 32 + (s & 3) * 8) * 2);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t o[4];
        e2m1x8_to_bf16(uint32_t(v.w[g][s >> 2][s & 3]), e[g][s >> 2], o);
        acc[g] = mfma_16x16x32_bf16(af, i32x4{int(o[0]), int(o[1]), int(o[2]), int(o[3])}, acc[g]);
      }
    }
  } else {
    f32x4 part[G];
#pragma unroll
    for (int g = 0; g < G; ++g) part[g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const i32x4 af = *reinterpret_cast<const i32x4*>(arow + (st * 128 + (s >> 1) * 64 + q * 16 + (s & 1) * 8) * 2);
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

// ---------------------------------------------------------------- gate / up

// LDS: tables | x rows [M][row_stride] | the routing's group scratch
__host__ __device__ inline uint32_t layer_row_stride(bool mx, int K) {
  const int st = mx ? 256 : 128;
  return uint32_t((K + st - 1) / st * st * 2 + 16);  // +16 B: rows read together fall in different banks
}

template <int WFMT, int LAY, int KPL>
__global__ __launch_bounds__(kLyThreads, 2) void moe_up_kernel(LayerArgs a) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  constexpr int D = kUpD;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int E = a.rt.E, R = a.M * a.rt.topk, H = int(a.H), I = int(a.I);
  const UpTables T = up_tables(smem, E, R);
  uint8_t* const xs = smem + up_table_bytes(E, R);

  // ---- the tokens' rows into LDS, zero-padded to whole steps
  const uint32_t stride = layer_row_stride(MX, H);
  const int chunks = int(stride / 16) - 1, valid = H / 8;
  for (int t = 0; t < a.M; ++t)
    for (int c = tid; c < chunks; c += kLyThreads) {
      i32x4 v = {0, 0, 0, 0};
      if (c < valid) v = *reinterpret_cast<const i32x4*>(a.x + (t + a.t0) * a.ldx + c * 8);
      *reinterpret_cast<i32x4*>(xs + t * stride + c * 16) = v;
    }
  build_tables<KPL>(a, T, reinterpret_cast<double*>(xs + a.M * stride));
  if (blockIdx.x == 0) {  // for the down stage
    const int rows = T.misc[0];
    for (int j = tid; j < rows; j += kLyThreads) a.rows[1 + j] = T.row[j];
    for (int e = tid; e < E; e += kLyThreads) a.rows[1 + 2 * R + e] = T.mask[e];
    if (tid == 0) a.rows[0] = rows;
  }

  // ---- items: (chosen expert, 16 gate + 16 up columns), dealt over the workgroups first.  The grid is
  // made for as many chosen experts as there can be; where tokens agree on a few, waves are left over,
  // and four or eight of a workgroup share an item, each a part of its K steps, at least two (us shared / not,
  // all tokens on the same experts: eight shares, FP8 7168 x 2048, 1 of 16 experts 74.8 / 81.8, MXFP4 7168 x
  // 512, 1 of 8 28.0 / 35.6; four, FP8 7168 x 512, 2 of 16 35.1 / 36.1, 2048 x 1024, 2 of 8 23.4 / 23.0; two,
  // FP8 4096 x 2048, 2 of 16 34.8 / 33.4, MXFP4 2880 x 2880, 4 of 32 31.1 / 30.0 -- MXFP4
  // tiled, 7168 x 2048, 4 of 32 40.9 / 42.6 is the one that gained -- so two do not share).  One token leaves
  // waves over only where masks leave it few experts.
  const WMat m = wmat<WFMT, LAY>(a.w1, a.s1, 2 * I, H);
  const int tiles = I / 16, total = __builtin_amdgcn_readfirstlane(T.misc[1]) * tiles;
  const int waves = int(gridDim.x) * kLyWaves;
  int KS = 1;
  while (KS < kLyWaves && 2 * KS * total <= waves && 4 * KS <= m.nsteps) KS *= 2;
  if (KS == 2) KS = 1;
  const int step = waves / KS;
  const int sub = wave & (KS - 1);
  const int st_lo = m.nsteps * sub / KS, st_hi = m.nsteps * (sub + 1) / KS;
  int item = (wave / KS) * int(gridDim.x) + int(blockIdx.x);
  if (KS == 1 && item >= total) return;
  auto geo_of = [&](int it) __attribute__((always_inline)) {
    WGeo<2> g;
    const int ti = it / tiles, nt = it - ti * tiles;
    const int e = __builtin_amdgcn_readfirstlane(T.touch[ti]);
    geo_expert(g, m, e);
    geo_group<WFMT, LAY, 2>(g, m, 0, nt);
    geo_group<WFMT, LAY, 2>(g, m, 1, tiles + nt);
    return g;
  };
  f32x4 acc[2];
  const uint8_t* arow = xs;
  int rows = 0, row0 = 0, nt = 0;
  float bg = 0.f, bu = 0.f;
  auto begin = [&]() __attribute__((always_inline)) {
    const int ti = item / tiles;
    nt = item - ti * tiles;
    const int ex = __builtin_amdgcn_readfirstlane(T.touch[ti]);
    rows = __builtin_amdgcn_readfirstlane(__popc(T.mask[ex]));
    row0 = __builtin_amdgcn_readfirstlane(T.start[ex]);
    arow = xs + uint32_t(T.row[row0 + min(l16, rows - 1)] & 0xff) * stride;
    acc[0] = acc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    // (requested here and waited for in finish(), behind all of the ring's requests made meanwhile)
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
      uint16_t hi = f2bf(h);
      // a finite h that rounds to infinity: bf16's largest value instead, the rest is in lo
      if ((hi & 0x7fffu) == 0x7f80u && fabsf(h) < __builtin_huge_valf()) --hi;
      const float hf = bf16f(hi);
      const uint16_t lo = f2bf(fabsf(hf) < __builtin_huge_valf() ? h - hf : 0.f);
      uint16_t* o = a.h + int64_t(row0 + i) * 2 * I + col;
      o[0] = hi;
      o[I] = lo;
    }
  };
  if (item < total) {
    // The ring: a pass over an item is padded to whole turns, so step i of every item sits in slot
    // i % D, and the last turn requests the next item's first steps (padding requests read nothing).
    // The code of an item's begin and end stands once: with a transition in every slot, a kernel
    // whose waves see a few steps each spent most of its time fetching instructions.
    const int n = st_hi - st_lo, npad = (n + D - 1) / D * D;
    WStep<WFMT, 2> ring[D];
    WGeo<2> cur = geo_of(item);
#pragma unroll
    for (int u = 0; u < D - 1; ++u) wload<WFMT, LAY, 2>(ring[u], cur, m, st_lo + u, st_hi);
    for (;;) {
      const int next = item + step;
      const bool more = next < total;
      const WGeo<2> nxt = geo_of(more ? next : item);
      begin();
      for (int s0 = 0; s0 < npad; s0 += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
          const int ls = s0 + u + D - 1;
          const bool nx = ls >= npad;
          wload<WFMT, LAY, 2>(ring[(u + D - 1) % D], geo_pick(nx, cur, nxt), m, st_lo + (nx ? ls - npad : ls),
                                nx && !more ? 0 : st_hi);
          if (s0 + u < n) wcompute<WFMT, LAY, 2>(acc, ring[u], arow, st_lo + s0 + u);
        }
      }
      if (KS > 1) break;  // (one item per wave at most)
      finish();
      if (!more) break;
      item = next;
      cur = nxt;
    }
  }
  if (KS > 1) {
    // the shares of an item meet in LDS, added in K order by the item's first wave
    f32x4* const sums = reinterpret_cast<f32x4*>(xs + a.M * stride);
    __syncthreads();  // the scratch's last reader is done
    sums[(wave * 2 + 0) * 64 + lane] = acc[0];
    sums[(wave * 2 + 1) * 64 + lane] = acc[1];
    __syncthreads();
    if (sub == 0 && item < total) {
      for (int k = 1; k < KS; ++k)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const f32x4 v = sums[((wave + k) * 2 + g) * 64 + lane];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[g][r] += v[r];
        }
      finish();
    }
  }
}


// ---------------------------------------------------------------- down

// The h rows of a step in registers on their way to LDS: the step's 256 (MXFP4) or 128 (FP8) columns of the
// hi and lo rows of a segment's kDownRows rows, 16 bytes per lane and read.
template <int WFMT>
struct HStep {
  static constexpr int N = WFMT == W_E2M1_MX ? kDownRows : kDownRows / 2;
  i32x4 v[N];
};

// What the lanes of a wave wrote to LDS before it, they read after it.  The LDS operations of a wave
// complete in order, so there is nothing to wait for: it holds the compiler to that order.
__device__ __forceinline__ void wave_handoff() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// LDS: tables | sums [2][slots][R][16] fp32 | h rows [8 waves][2 kDownRows][step columns] bf16
__host__ __device__ inline int down_sum_rows(int R) {
  // segments that many waves share: fewer than eight segments of at most kDownRows rows, eight
  // shares each; else two shares of every row
  return R * 2 > 7 * kDownRows * 8 ? R * 2 : 7 * kDownRows * 8;
}

template <int WFMT, int LAY>
__global__ __launch_bounds__(kLyThreads, 2) void moe_down_kernel(LayerArgs a) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  constexpr int D = kDownD, SE = MX ? 256 : 128, ROWB = SE * 2;  // columns of a step, bytes of its rows in LDS
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int topk = a.rt.topk, R = a.M * topk, H = int(a.H), I = int(a.I);
  const DownTables T = down_tables(smem, R);
  const int sum_rows = down_sum_rows(R);
  float* const sums = reinterpret_cast<float*>(smem + down_table_bytes(R));
  uint8_t* const hs = smem + down_table_bytes(R) + uint32_t(sum_rows) * 2 * 64 + uint32_t(wave) * (2 * kDownRows * ROWB);
  const WMat m = wmat<WFMT, LAY>(a.w2, a.s2, H, I);
  const int items = H / 16;

  // ---- tables
  const int rows = __builtin_amdgcn_readfirstlane(a.rows[0]);
  for (int r = tid; r < R; r += kLyThreads) T.pos[r] = a.rows[1 + R + r];
  if (wave == 0) {
    int n = 0;
    for (int r0 = 0; r0 < rows; r0 += 64) {
      const int j = r0 + lane;
      bool first = false;
      int e = 0;
      if (j < rows) {
        // an expert's rows are cut every kDownRows: row j opens a segment when its distance from
        // its expert's first row is a multiple of that
        const int v = a.rows[1 + j];
        e = v >> 8;
        const int d = __popc(a.rows[1 + 2 * R + e] & ((1 << (v & 0xff)) - 1));
        first = d % kDownRows == 0;
      }
      const uint64_t mk = __ballot(first);
      const int at = n + __popcll(mk & ((uint64_t(2) << lane) - 1)) - 1;
      if (j < rows) T.segof[j] = at;
      if (first) T.seg[at] = e << 16 | j;
      n += __popcll(mk);
    }
    if (lane == 0) *T.misc = n;
  }
  __syncthreads();
  const int nseg = __builtin_amdgcn_readfirstlane(*T.misc);
  const int tok = tid >> 4, tc = tid & 15;
  const int my = items > int(blockIdx.x) ? (items - 1 - int(blockIdx.x)) / int(gridDim.x) + 1 : 0;
  if (nseg == 0) {  // no token has an expert
    for (int i = 0; i < my; ++i)
      if (tok < a.M) a.out[(tok + a.t0) * a.ldo + (int64_t(blockIdx.x) + int64_t(i) * gridDim.x) * 16 + tc] = 0;
    return;
  }
  if (my == 0) return;

  // ---- this wave's share of every item: steps [lo, hi) of the segments' nsteps each
  const int S = nseg * m.nsteps;
  const bool few = S < kLyWaves;  // one step per wave
  const int lo = few ? min(wave, S) : S * wave / kLyWaves, hi = few ? min(wave + 1, S) : S * (wave + 1) / kLyWaves;
  auto wave_of = [&](int step) __attribute__((always_inline)) { return few ? step : (kLyWaves * (step + 1) - 1) / S; };
  auto seg_at = [&](int sg) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(T.seg[sg]); };
  auto seg_end = [&](int sg) __attribute__((always_inline)) {
    return sg + 1 < nseg ? __builtin_amdgcn_readfirstlane(T.seg[sg + 1]) & 0xffff : rows;
  };

  const uint8_t* const hp = reinterpret_cast<const uint8_t*>(a.h);
  const uint32_t h_bytes = uint32_t(rows) * uint32_t(I) * 4u;
  const __amdgpu_buffer_rsrc_t hb = raw_buffer(hp, h_bytes);
  const int kl = (lane & (SE / 8 - 1)) * 8;  // this lane's first column of a step's h rows
  const bool hpast = (m.nsteps - 1) * SE + kl >= I;

  // The share is walked in parts: steps [st, st + n) of one segment, for one item.
  struct Part {
    int ci, p;            // item (count), position in [lo, hi)
    int seg, st, n;
    int row0, sm;         // the segment's first sorted row, its rows
  };
  auto part_at = [&](int ci, int p) __attribute__((always_inline)) {
    Part o;
    o.ci = ci;
    o.p = p;
    o.seg = p / m.nsteps;
    o.st = p - o.seg * m.nsteps;
    o.n = min(m.nsteps - o.st, hi - p);
    o.row0 = seg_at(o.seg) & 0xffff;
    o.sm = seg_end(o.seg) - o.row0;
    return o;
  };
  struct Geo {
    WGeo<1> w;
    uint32_t h[HStep<WFMT>::N];
  };
  auto geo_of = [&](const Part& o) __attribute__((always_inline)) {
    Geo g;
    geo_expert(g.w, m, seg_at(o.seg) >> 16);
    geo_group<WFMT, LAY, 1>(g.w, m, 0, int(blockIdx.x) + o.ci * int(gridDim.x));
#pragma unroll
    for (int i = 0; i < HStep<WFMT>::N; ++i) {
      // rows of 32 (MXFP4) or 16 (FP8) chunks: hi row, lo row (, the next row's hi and lo)
      const int r = MX ? i : 2 * i + (lane >> 5), half = MX ? lane >> 5 : (lane >> 4) & 1;
      g.h[i] = r < o.sm ? (uint32_t(o.row0 + r) * 2u + uint32_t(half)) * uint32_t(I) * 2u + uint32_t(kl) * 2u : kNoRead;
    }
    return g;
  };
  WStep<WFMT, 1> ring[D];
  HStep<WFMT> hring[D];
  auto load = [&](int slot, const WGeo<1>& w, const uint32_t* h0, const uint32_t* h1, bool nx, int st, int st_end)
      __attribute__((always_inline)) {
    wload<WFMT, LAY, 1>(ring[slot], w, m, st, st_end);
    const bool no = st >= st_end || (MX && st == m.nsteps - 1 && hpast);
    const int ho = st >= st_end ? 0 : st * (SE * 2);
#pragma unroll
    for (int i = 0; i < HStep<WFMT>::N; ++i)
      hring[slot].v[i] = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(hb, no ? kNoRead : (nx ? h1[i] : h0[i]), ho, 0));
  };

  // the item's rows are summed: each token's in the order of its experts, a row's shares in K order.
  // One barrier an item: the sums of the next one go to the other half.
  auto end_item = [&](int ci) __attribute__((always_inline)) {
    __syncthreads();
    if (tok < a.M) {
      float s = 0.f;
      for (int k = 0; k < topk; ++k) {
        const int j = T.pos[tok * topk + k];
        if (j < 0) continue;
        const int s0 = T.segof[j] * m.nsteps, w0 = wave_of(s0), w1 = wave_of(s0 + m.nsteps - 1);
        const float* p = sums + ((ci & 1) * sum_rows + j) * 16 + tc;
        float y = 0.f;
        for (int w = 0; w <= w1 - w0; ++w) y += p[w * rows * 16];
        s += y;
      }
      a.out[(tok + a.t0) * a.ldo + (int64_t(blockIdx.x) + int64_t(ci) * gridDim.x) * 16 + tc] = f2bf(s);
    }
  };

  if (hi <= lo) {  // a wave without a share only joins the sums
    for (int ci = 0; ci < my; ++ci) end_item(ci);
    return;
  }
  Part cp = part_at(0, lo);
  Geo cg = geo_of(cp);
#pragma unroll
  for (int u = 0; u < D - 1; ++u) load(u, cg.w, cg.h, cg.h, false, cp.st + u, cp.st + cp.n);
  for (;;) {
    const bool item_ends = cp.p + cp.n == hi;
    const bool more = !item_ends || cp.ci + 1 < my;
    const Part np = more ? part_at(item_ends ? cp.ci + 1 : cp.ci, item_ends ? lo : cp.p + cp.n) : cp;
    const Geo ng = geo_of(np);
    const int npad = (cp.n + D - 1) / D * D, nend = more ? np.st + np.n : 0;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    // MFMA rows i and i + 8 are the hi and lo terms of the segment's row i; LDS row 2 i + term
    const RowAt<WFMT> at = row_at<WFMT>(hs, 2 * ((l16 & 7) < cp.sm ? (l16 & 7) : 0) + (l16 >> 3));
    for (int s0 = 0; s0 < npad; s0 += D) {
#pragma unroll
      for (int u = 0; u < D; ++u) {
        const int ls = s0 + u + D - 1;
        const bool nx = ls >= npad;
        load((u + D - 1) % D, geo_pick(nx, cg.w, ng.w), cg.h, ng.h, nx, nx ? np.st + ls - npad : cp.st + ls,
             nx ? nend : cp.st + cp.n);
        if (s0 + u < cp.n) {
          // the step's h rows into this wave's LDS rows (16-byte chunk c of LDS row r in slot c ^ r)
#pragma unroll
          for (int i = 0; i < HStep<WFMT>::N; ++i) {
            const int r = MX ? 2 * i + (lane >> 5) : 4 * i + (lane >> 4);
            *reinterpret_cast<i32x4*>(hs + r * ROWB + (((lane & (SE / 8 - 1)) ^ r) * 16)) = hring[u].v[i];
          }
          wave_handoff();
          wcompute_rows<WFMT, LAY>(acc, ring[u], at);
          wave_handoff();  // before the next step's rows
        }
      }
    }
    {
      const int slot = wave - wave_of(cp.seg * m.nsteps);
      float* p = sums + (((cp.ci & 1) * sum_rows) + slot * rows + cp.row0) * 16 + l16;
      f32x4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = acc[r] + __shfl_xor(acc[r], 32, kWave);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 4 * q + r;
        if (q < 2 && i < cp.sm) p[i * 16] = o[r];
      }
    }
    if (item_ends) end_item(cp.ci);
    if (!more) break;
    cp = np;
    cg = ng;
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

// the shares of items (2 x 16 x 16 fp32 per wave), or before them the routing's group scratch
// (E doubles per wave)
uint32_t up_scratch(int E) { return std::max(uint32_t(kLyWaves * 2 * 256 * 4), uint32_t(kLyWaves * E * 8)); }

uint32_t up_lds(bool mx, int64_t H, int E, int topk, int M) {
  return up_table_bytes(E, M * topk) + uint32_t(M) * layer_row_stride(mx, int(H)) + up_scratch(E);
}

uint32_t down_lds(bool mx, int R) {
  return down_table_bytes(R) + uint32_t(down_sum_rows(R)) * 2 * 64 + uint32_t(kLyWaves * 2 * kDownRows * (mx ? 512 : 256));
}

template <int WFMT, int LAY>
void launch_layer_t(const LayerArgs& a, hipStream_t st) {
  constexpr bool MX = WFMT == W_E2M1_MX;
  const int R = a.M * a.rt.topk;
  const int64_t most = std::min<int64_t>(a.rt.E, R);  // chosen experts at most
  const unsigned gu = unsigned(std::min<int64_t>(layer_cus(), cdiv(most * (a.I / 16), kLyWaves)));
  const size_t lu = up_lds(MX, a.H, a.rt.E, a.rt.topk, a.M);
  if (a.rt.E <= 128)
    hipLaunchKernelGGL((moe_up_kernel<WFMT, LAY, 2>), dim3(gu), dim3(kLyThreads), lu, st, a);
  else if (a.rt.E <= 256)
    hipLaunchKernelGGL((moe_up_kernel<WFMT, LAY, 4>), dim3(gu), dim3(kLyThreads), lu, st, a);
  else
    hipLaunchKernelGGL((moe_up_kernel<WFMT, LAY, 8>), dim3(gu), dim3(kLyThreads), lu, st, a);
  const unsigned gd = unsigned(std::min<int64_t>(layer_cus(), a.H / 16));
  hipLaunchKernelGGL((moe_down_kernel<WFMT, LAY>), dim3(gd), dim3(kLyThreads), down_lds(MX, R), st, a);
}
}  // namespace

int layer_pass_tokens(int wfmt, int64_t H, int32_t E, int32_t topk) {
  const bool mx = wfmt == W_E2M1_MX;
  int m = kLayerMaxTokens;
  while (m > 0 && std::max(up_lds(mx, H, E, topk, m), down_lds(mx, m * topk)) > kLyMaxLds) --m;
  return m;
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
    if (a.wfmt == W_E2M1_MX) {
      const bool pairs = a.H % 64 == 0 && a.I % 64 == 0 &&
                         ((reinterpret_cast<uintptr_t>(a.s1) | reinterpret_cast<uintptr_t>(a.s2)) & 1) == 0;
      if (a.tiled) launch_layer_t<W_E2M1_MX, kTiled>(a, st);
      else if (pairs) launch_layer_t<W_E2M1_MX, kPlainPairs>(a, st);
      else launch_layer_t<W_E2M1_MX, kPlain>(a, st);
    } else {
      if (a.tiled) launch_layer_t<W_E4M3_BLOCK, kTiled>(a, st);
      else launch_layer_t<W_E4M3_BLOCK, kPlain>(a, st);
    }
  }
}

}  // namespace mxq
