// Expert routing: router logits [M, E] -> expert ids and weights [M, topk] (route_common.hpp holds
// the formulas).  One wave per token, four tokens per workgroup; many tokens take 16 lanes each, where
// the groups allow it.  Scores are computed in fp32; where picks that decide the result lie closer than
// fp32 scores can tell apart, the wave repeats its token in 64 bits, so the chosen experts and their
// order are those of 64-bit scores.  How many tokens that is depends on the router: 16384 x 256 in 8
// groups, sigmoid scores, take 19 us with ordinary biases, and without any 21, 35 and 56 us as the
// logits' deviation grows over 2, 4 and 8 (at 8 most scores are 0 or 1 to fp32).
#include "layer.hpp"
#include "route_common.hpp"

namespace mxq {

namespace {
constexpr int kRouteWaves = 4;
// From here on 16 lanes per token (us, against a wave per token; 256 experts in 8 groups: 16384 tokens
// 19.3 / 35.9, 4096 13.0 / 14.8, 2048 12.9 / 13.4, 1024 11.3 / 11.1, most of it one token repeated in
// 64 bits; 128 experts: 16384 tokens 5.7 / 11.6, 1024 4.7 / 4.7).
constexpr int64_t kRouteRowsFrom = 1024;
}

template <int KPL, bool BF16>
__global__ __launch_bounds__(256) void moe_route_kernel(const void* __restrict__ logits, int64_t M, int64_t ld,
                                                        RouteArgs a, int32_t* __restrict__ ids,
                                                        float* __restrict__ weights) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double* const s_val = reinterpret_cast<double*>(smem) + int64_t(wave) * a.E;
  const int64_t t = int64_t(blockIdx.x) * kRouteWaves + wave;
  if (t >= M) return;
  float l[KPL], b[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane * KPL + i;
    l[i] = -__builtin_huge_valf();
    b[i] = 0.f;
    if (e < a.E) {
      l[i] = BF16 ? bf16f(reinterpret_cast<const uint16_t*>(logits)[t * ld + e])
                  : reinterpret_cast<const float*>(logits)[t * ld + e];
      if (a.bias) b[i] = a.bias[e];
    }
  }
  bool close;
  RouteSlot s = route_token<KPL, float>(l, b, a, reinterpret_cast<float*>(s_val), close);
  if (close) {
    bool unused;
    s = route_token<KPL, double>(l, b, a, s_val, unused);
  }
  if (lane < a.topk) {
    ids[t * a.topk + lane] = s.id;
    weights[t * a.topk + lane] = s.w;
  }
}

// ---------------------------------------------------------------- many tokens

// Many tokens are bound by instructions, and a wave's 64 lanes on one token repeat most of them
// (reductions, branches, the chosen expert's broadcast).  Here 16 lanes take a token, four tokens a
// wave; lane j holds experts [j KPL, (j + 1) KPL).  A selection round is a maximum over the lane's
// registers, one over its 16-lane row, and the minimum of the indices that hold it.  The chosen logits
// are read again for the weights.  Tokens with picks too close for fp32 are repeated by the whole
// wave in 64 bits, one after the other.
template <int CTRL>
__device__ __forceinline__ float row_ror(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, row_ror<0x128>(v));  // rotate by 8, 4, 2, 1 within 16 lanes
  v = fmaxf(v, row_ror<0x124>(v));
  v = fmaxf(v, row_ror<0x122>(v));
  return fmaxf(v, row_ror<0x121>(v));
}
__device__ __forceinline__ float row_total(float v) {
  v += row_ror<0x128>(v);
  v += row_ror<0x124>(v);
  v += row_ror<0x122>(v);
  return v + row_ror<0x121>(v);
}
__device__ __forceinline__ int row_min(int v) {
  v = min(v, __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, true));
  v = min(v, __builtin_amdgcn_update_dpp(0, v, 0x124, 0xf, 0xf, true));
  v = min(v, __builtin_amdgcn_update_dpp(0, v, 0x122, 0xf, 0xf, true));
  return min(v, __builtin_amdgcn_update_dpp(0, v, 0x121, 0xf, 0xf, true));
}

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* logits, int64_t i) {
  return BF16 ? bf16f(reinterpret_cast<const uint16_t*>(logits)[i]) : reinterpret_cast<const float*>(logits)[i];
}

// VEC: E % 4 == 0 and rows (and the bias) aligned to four elements.  lpg: lanes of a group (0: no groups).
template <int KPL, bool BF16, bool VEC>
__global__ __launch_bounds__(256) void moe_route_rows_kernel(const void* __restrict__ logits, int64_t M, int64_t ld,
                                                             RouteArgs a, int lpg, int32_t* __restrict__ ids,
                                                             float* __restrict__ weights) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & 15;
  const int64_t t0 = (int64_t(blockIdx.x) * kRouteWaves + wave) * 4;
  if (t0 >= M) return;
  const int64_t t = min(t0 + (lane >> 4), M - 1);  // (a repeated last token is not written)
  const float kNone = -__builtin_huge_valf();
  const bool by_score = a.bias != nullptr;

  float l[KPL], pick[KPL];
#pragma unroll
  for (int i = 0; i < KPL; i += 4) {
    const int e = j * KPL + i;
#pragma unroll
    for (int d = 0; d < 4; ++d) l[i + d] = kNone;
    if (VEC) {
      if (e < a.E) {
        if (BF16) {
          const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(logits) + t * ld + e);
          l[i] = __uint_as_float(v.x << 16);
          l[i + 1] = __uint_as_float(v.x & 0xffff0000u);
          l[i + 2] = __uint_as_float(v.y << 16);
          l[i + 3] = __uint_as_float(v.y & 0xffff0000u);
        } else {
          const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(logits) + t * ld + e);
          l[i] = v.x;
          l[i + 1] = v.y;
          l[i + 2] = v.z;
          l[i + 3] = v.w;
        }
      }
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if (e + d < a.E) l[i + d] = logit_at<BF16>(logits, t * ld + e + d);
    }
  }

  // ---- scores (as route_token; sigmoids with the fast exponential and reciprocal, whose errors
  // route_err covers)
  float lmax = kNone, sum = 1.f;
  const bool need_p = by_score || (lpg && a.group_top2) || !a.renormalize;
  if (!a.sigmoid && need_p) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) lmax = fmaxf(lmax, l[i]);  // (fmaxf drops a NaN)
    lmax = row_max(lmax);
  }
#pragma unroll
  for (int i = 0; i < KPL; ++i) pick[i] = l[i] > kNone ? l[i] : kNone;
  bool scores = false;  // pick holds scores: the fp32 border may be close
  if (need_p && a.sigmoid) {
    if (by_score || (lpg && a.group_top2)) {
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        l[i] = l[i] > kNone ? __builtin_amdgcn_rcpf(1.f + __expf(-l[i])) : 0.f;
    }
  } else if (need_p) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      l[i] = l[i] > kNone ? (l[i] == lmax ? 1.f : expf(l[i] - lmax)) : 0.f;
      s += l[i];
    }
    sum = fmaxf(1.f, row_total(s));
    const float inv = 1.f / sum;
#pragma unroll
    for (int i = 0; i < KPL; ++i) l[i] *= inv;
  }
  if (by_score) {
    scores = true;
#pragma unroll
    for (int i = 0; i < KPL; i += 4) {
      const int e = j * KPL + i;
      float b[4] = {0.f, 0.f, 0.f, 0.f};
      if (VEC) {
        if (e < a.E) {
          const float4 v = *reinterpret_cast<const float4*>(a.bias + e);
          b[0] = v.x;
          b[1] = v.y;
          b[2] = v.z;
          b[3] = v.w;
        }
      } else {
#pragma unroll
        for (int d = 0; d < 4; ++d)
          if (e + d < a.E) b[d] = a.bias[e + d];
      }
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const float v = l[i + d] + b[d];
        pick[i + d] = pick[i + d] > kNone && v > kNone ? v : kNone;
      }
    }
  }

  // ---- groups of lpg lanes
  bool close = false;
  if (lpg) {
    float m1 = kNone, m2 = kNone;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const float x = (!a.group_top2 || by_score) ? pick[i] : (pick[i] > kNone ? l[i] : kNone);
      m2 = fmaxf(m2, fminf(m1, x));
      m1 = fmaxf(m1, x);
    }
    for (int o = 1; o < lpg; o <<= 1) {
      const float o1 = __shfl_xor(m1, o, kWave), o2 = __shfl_xor(m2, o, kWave);
      m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
      m1 = fmaxf(m1, o1);
    }
    const int mine = j / lpg;
    if (mine >= a.n_group) m1 = m2 = kNone;
    float gs = a.group_top2 && m2 > kNone ? m1 + m2 : m1;
    bool keep = false;
    for (int r = 0; r < a.topk_group; ++r) {
      const float mx = row_max(gs);
      const int g = row_min(gs == mx && mx > kNone ? mine : 64);
      if (g == mine) {
        keep = true;
        gs = kNone;
      }
    }
    if (by_score || a.group_top2) {
      const RouteBounds bd = route_bounds(m1, a.group_top2 ? m2 : kNone, a.sigmoid);
      const float out = row_max(keep ? kNone : bd.hi), in = -row_max(keep ? -bd.lo : kNone);
      close = out > kNone && !(out < in);
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i) pick[i] = keep ? pick[i] : kNone;
  }

  // ---- the topk largest picks
  int id = -1;
  float last = kNone;
  for (int k = 0; k < a.topk + (scores ? 1 : 0); ++k) {
    float best = pick[0];
#pragma unroll
    for (int i = 1; i < KPL; ++i) best = fmaxf(best, pick[i]);
    const float mx = row_max(best);
    const bool any = mx > kNone;
    if (!__any(any)) break;
    if (scores && k > 0 && any) close = close || route_near(last, mx, a.sigmoid);
    last = mx;
    if (k == a.topk) break;
    int at = 1 << 20;
#pragma unroll
    for (int i = KPL - 1; i >= 0; --i) at = pick[i] == mx ? i : at;
    const int e = row_min(at + j * KPL);
    if (any && j == k) id = e;
    const int d = e - j * KPL;
#pragma unroll
    for (int i = 0; i < KPL; ++i) pick[i] = d == i ? kNone : pick[i];
  }

  // ---- weights
  const float my_l = id >= 0 ? logit_at<BF16>(logits, t * ld + id) : kNone;
  float w = 0.f;
  if (a.renormalize) {
    const float m = row_max(my_l);
    const float v = id >= 0 ? route_ratio<float>(my_l, m, a.sigmoid) : 0.f;
    const float tot = row_total(v);
    if (id >= 0) w = v / tot * a.scale;
  } else if (id >= 0) {
    w = (a.sigmoid ? 1.f / (1.f + expf(-my_l)) : (my_l == lmax ? 1.f : expf(my_l - lmax)) / sum) * a.scale;
  }
  const uint64_t again = __ballot(close);
  if (!close && t0 + (lane >> 4) < M && j < a.topk) {
    ids[t * a.topk + j] = id;
    weights[t * a.topk + j] = w;
  }
  if (again == 0) return;
  constexpr int WPL = KPL >= 4 ? KPL / 4 : 1;
  for (int r = 0; r < 4; ++r) {
    if (((again >> (16 * r)) & 1) == 0 || t0 + r >= M) continue;
    float wl[WPL], wb[WPL];
#pragma unroll
    for (int i = 0; i < WPL; ++i) {
      const int e = lane * WPL + i;
      wl[i] = e < a.E ? logit_at<BF16>(logits, (t0 + r) * ld + e) : kNone;
      wb[i] = e < a.E && a.bias ? a.bias[e] : 0.f;
    }
    bool unused;
    const RouteSlot s =
        route_token<WPL, double>(wl, wb, a, reinterpret_cast<double*>(smem) + int64_t(wave) * a.E, unused);
    if (lane < a.topk) {
      ids[(t0 + r) * a.topk + lane] = s.id;
      weights[(t0 + r) * a.topk + lane] = s.w;
    }
  }
}

void launch_moe_route(const void* logits, bool bf16, int64_t M, int64_t ld, const RouteArgs& a, int32_t* ids,
                      float* weights, hipStream_t stream) {
  if (M <= 0) return;
  const dim3 grid{unsigned(cdiv(M, kRouteWaves))}, block{256u};
  const size_t lds = a.n_group > 1 ? size_t(kRouteWaves) * a.E * 8 : 0;
  // Lane j of 16 holds kpl experts, by E alone, so a group has to be one, two, four, ... lanes: 160
  // experts in 8 groups of 20, for one, stay with a wave per token.
  if (M >= kRouteRowsFrom && a.topk <= 16) {
    const int kpl = a.E <= 64 ? 4 : (a.E <= 128 ? 8 : (a.E <= 256 ? 16 : 32));
    const int lpg = a.n_group > 1 ? a.group_size / kpl : 0;
    if (a.n_group == 1 || (lpg > 0 && a.group_size % kpl == 0 && (lpg & (lpg - 1)) == 0)) {
      const size_t esz = bf16 ? 2 : 4;
      const bool vec = a.E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % (4 * esz) == 0 &&
                       reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
      const dim3 rows{unsigned(cdiv(M, 4 * kRouteWaves))};
#define MXQ_RR(K, B, V) \
  hipLaunchKernelGGL((moe_route_rows_kernel<K, B, V>), rows, block, lds, stream, logits, M, ld, a, lpg, ids, weights)
#define MXQ_RR_T(K)                            \
  do {                                         \
    if (bf16 && vec) MXQ_RR(K, true, true);    \
    else if (bf16) MXQ_RR(K, true, false);     \
    else if (vec) MXQ_RR(K, false, true);      \
    else MXQ_RR(K, false, false);              \
  } while (0)
      if (kpl == 4) MXQ_RR_T(4);
      else if (kpl == 8) MXQ_RR_T(8);
      else if (kpl == 16) MXQ_RR_T(16);
      else MXQ_RR_T(32);
#undef MXQ_RR_T
#undef MXQ_RR
      return;
    }
  }
#define MXQ_RT(KPL)                                                                                             \
  do {                                                                                                          \
    if (bf16)                                                                                                   \
      hipLaunchKernelGGL((moe_route_kernel<KPL, true>), grid, block, lds, stream, logits, M, ld, a, ids, weights);  \
    else                                                                                                        \
      hipLaunchKernelGGL((moe_route_kernel<KPL, false>), grid, block, lds, stream, logits, M, ld, a, ids, weights); \
  } while (0)
  if (a.E <= 64) MXQ_RT(1);
  else if (a.E <= 128) MXQ_RT(2);
  else if (a.E <= 256) MXQ_RT(4);
  else MXQ_RT(8);
#undef MXQ_RT
}

}  // namespace mxq
