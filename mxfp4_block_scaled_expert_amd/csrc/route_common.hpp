// Routing of one token by one wave: router logits -> the token's experts and their weights.
//
//   live(e)   l[e] > -inf (a NaN or -inf logit takes its expert out)
//   p[e]      softmax: exp(l[e] - max l) / sum over live experts;  sigmoid: 1 / (1 + exp(-l[e]))
//   pick[e]   p[e] + bias[e] with a correction bias, else l[e] (p is monotone in l)
//   groups    E / n_group consecutive experts each; a group's score is its largest pick, or the sum
//             of its two largest p + bias; only the topk_group best groups stay
//   chosen    the topk largest picks, largest first, equal picks by the lower index; slots that
//             find no live expert get id -1 and weight 0
//   weight    p of the chosen expert, divided by the chosen experts' sum when renormalising
//             (as a ratio of exponentials, so it does not depend on how small the p are), times scale
//
// Lane l holds experts [l * KPL, (l + 1) * KPL): a round of the selection is one wave-wide maximum
// of the lanes' best picks, and the lowest lane that holds it is the lowest index.
#pragma once

#include "layer.hpp"

namespace mxq {

// ---------------------------------------------------------------- wave reductions (result in every lane)

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f(float old, float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, ROWS, 0xf, false));
}

__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_f<0x111, 0xf>(v, v));  // row_shr:1, 2, 4, 8: lane 15 of a row holds the row's maximum
  v = fmaxf(v, dpp_f<0x112, 0xf>(v, v));
  v = fmaxf(v, dpp_f<0x114, 0xf>(v, v));
  v = fmaxf(v, dpp_f<0x118, 0xf>(v, v));
  v = fmaxf(v, dpp_f<0x142, 0xa>(v, v));  // row_bcast:15 into rows 1 and 3
  v = fmaxf(v, dpp_f<0x143, 0xc>(v, v));  // row_bcast:31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ float wave_total(float v) {
  v += dpp_f<0x111, 0xf>(0.f, v);
  v += dpp_f<0x112, 0xf>(0.f, v);
  v += dpp_f<0x114, 0xf>(0.f, v);
  v += dpp_f<0x118, 0xf>(0.f, v);
  v += dpp_f<0x142, 0xa>(0.f, v);
  v += dpp_f<0x143, 0xc>(0.f, v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// The same for 64-bit values, as two 32-bit moves a step (through LDS shuffles a routing in 64 bits
// took 9 us more).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_d(double old, double v) {
  const int lo = __builtin_amdgcn_update_dpp(__double2loint(old), __double2loint(v), CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(__double2hiint(old), __double2hiint(v), CTRL, ROWS, 0xf, false);
  return __hiloint2double(hi, lo);
}
__device__ __forceinline__ double lane_value(double v, int src) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), src),
                          __builtin_amdgcn_readlane(__double2loint(v), src));
}

__device__ __forceinline__ double wave_max(double v) {
  v = fmax(v, dpp_d<0x111, 0xf>(v, v));
  v = fmax(v, dpp_d<0x112, 0xf>(v, v));
  v = fmax(v, dpp_d<0x114, 0xf>(v, v));
  v = fmax(v, dpp_d<0x118, 0xf>(v, v));
  v = fmax(v, dpp_d<0x142, 0xa>(v, v));
  v = fmax(v, dpp_d<0x143, 0xc>(v, v));
  return lane_value(v, 63);
}

__device__ __forceinline__ double wave_total(double v) {
  v += dpp_d<0x111, 0xf>(0., v);
  v += dpp_d<0x112, 0xf>(0., v);
  v += dpp_d<0x114, 0xf>(0., v);
  v += dpp_d<0x118, 0xf>(0., v);
  v += dpp_d<0x142, 0xa>(0., v);
  v += dpp_d<0x143, 0xc>(0., v);
  return lane_value(v, 63);
}

// Lane `src`'s value (src uniform) in every lane.
__device__ __forceinline__ float lane_value(float v, int src) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), src));
}

__device__ __forceinline__ float route_exp(float x) { return expf(x); }
__device__ __forceinline__ double route_exp(double x) { return exp(x); }

// What an fp32 score p is off by at most, with u = 2^-24 a rounding.  sigmoid: the exponential (4 u of
// itself; by the fast instruction (2 |l| + 2) u), the sum and the reciprocal leave p (1 - p) (2 |l| + 2) u +
// 3 p u < 4 u: 2^-21 is twice that.  softmax: d = max l - l is rounded (d u of the exponential), the
// exponential is 4 u, the sum of at most 512 of them 35 u and their own errors' mean, which is at most
// (ln 512 + 4) u, then two more: together all scores of a token are off by less than 58 u, so 32 u for
// either side of a comparison cover it.
__device__ __forceinline__ float route_err(int sigmoid, int scores) {
  return sigmoid ? float(scores) * 0x1p-21f : 0x1p-19f;
}

// Whether picks p + b may be in another order than fp32 has them, x first: each carries its score's
// error and a rounding of itself (2^-22 leaves four).  A pick's error grows slower than the pick, so
// looking at neighbours in the order is enough.
__device__ __forceinline__ bool route_near(float x, float y, int sigmoid) {
  return !(x - y > 2.f * route_err(sigmoid, 1) + 0x1p-22f * (fabsf(x) + fabsf(y)));
}

// The bounds of a group's score from its two largest terms (m2: -inf if only one counts).  Here it is
// the terms' sizes that say what was rounded: m1 and m2 may nearly cancel, so every group has its own
// error and no order of groups bounds it.  A sum that overflowed may be anything; an infinite
// term (an infinite bias) is exact.
struct RouteBounds {
  float lo, hi;
};
__device__ __forceinline__ RouteBounds route_bounds(float m1, float m2, int sigmoid) {
  const float inf = __builtin_huge_valf();
  const bool two = m2 > -inf;
  if (!(m1 > -inf) || m1 == inf) return {m1, m1};
  const float v = two ? m1 + m2 : m1, mag = two ? fabsf(m1) + fabsf(m2) : fabsf(m1);
  if (!(mag < inf)) return {-inf, inf};
  const float e = route_err(sigmoid, two ? 2 : 1) + 0x1p-22f * mag;
  return {v - e, v + e};
}

// A chosen expert's score relative to that of the largest chosen logit m, which is what
// renormalising divides.  softmax: exp(l - m).  sigmoid: exp(-log(1 + exp(-l))) relative to m's, so
// that tiny scores keep their ratio.
template <typename T>
__device__ __forceinline__ T route_ratio(float l, float m, int sigmoid) {
  if (l == m) return T(1);
  if (sigmoid && m > 0.f) return (T(1) + route_exp(-T(m))) / (T(1) + route_exp(-T(l)));
  const T ratio = route_exp(T(l) - T(m));  // exp(l) / exp(m)
  return sigmoid ? ratio * (T(1) + route_exp(T(m))) / (T(1) + route_exp(T(l))) : ratio;
}

// What lane k < topk holds after a routing: slot k's expert (-1: none) and weight.
struct RouteSlot {
  int32_t id;
  float w;
};

// One token.  l[i]: this lane's logits (-inf past E).  b[i]: their correction bias (0 without
// one).  T: the arithmetic of the scores.  s_val: T[E] of LDS of this wave's own (groups only).
// `close` is set when two picks that decide the result are nearer than fp32 scores can tell
// apart (T = float with scores in the comparison only); the caller then repeats the token in
// 64 bits.
template <int KPL, typename T>
__device__ __forceinline__ RouteSlot route_token(const float (&l)[KPL], const float (&b)[KPL], const RouteArgs& a,
                                                 T* s_val, bool& close) {
  const int lane = threadIdx.x & 63;
  const T kNone = T(-__builtin_huge_valf());
  constexpr bool F32 = sizeof(T) == 4;

  // ---- scores
  float lmax = -__builtin_huge_valf();
  bool live[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    live[i] = l[i] > -__builtin_huge_valf();
    if (live[i]) lmax = fmaxf(lmax, l[i]);
  }
  const bool by_score = a.bias != nullptr;                      // picks are p + bias
  const bool grouped = a.n_group > 1;
  const bool need_p = by_score || (grouped && a.group_top2) || !(a.renormalize);
  T p[KPL];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) p[i] = live[i] && need_p ? T(1) / (T(1) + route_exp(-T(l[i]))) : T(0);
  } else {
    lmax = wave_max(lmax);
    T sum = T(0);
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      // (l == lmax covers +inf, whose share the +inf experts split evenly)
      p[i] = live[i] && need_p ? (l[i] == lmax ? T(1) : route_exp(T(l[i]) - T(lmax))) : T(0);
      sum += p[i];
    }
    if (need_p) {
      const T inv = T(1) / fmax(T(1), wave_total(sum));  // a token with a live expert sums to at least 1
#pragma unroll
      for (int i = 0; i < KPL; ++i) p[i] *= inv;
    }
  }
  T pick[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const T v = by_score ? p[i] + T(b[i]) : T(l[i]);
    pick[i] = live[i] && v > kNone ? v : kNone;  // (a NaN bias takes its expert out too)
  }
  close = false;

  // ---- groups
  if (grouped) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int e = lane * KPL + i;
      if (e < a.E) s_val[e] = (!a.group_top2 || by_score) ? pick[i] : (pick[i] > kNone ? p[i] : kNone);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    T gs = kNone, m1 = kNone, m2 = kNone;
    if (lane < a.n_group) {
      const T* v = s_val + lane * a.group_size;
#pragma unroll 8  // reads in flight together
      for (int j = 0; j < a.group_size; ++j) {
        const T x = v[j];
        m2 = fmax(m2, fmin(m1, x));
        m1 = fmax(m1, x);
      }
      gs = a.group_top2 && m2 > kNone ? m1 + m2 : m1;
    }
    uint64_t keep = 0;
    for (int r = 0; r < a.topk_group; ++r) {
      const T mx = wave_max(gs);
      if (!(mx > kNone)) break;
      const int g = __builtin_ctzll(__ballot(gs == mx));
      keep |= uint64_t(1) << g;
      if (lane == g) gs = kNone;
    }
    if (F32 && (by_score || a.group_top2)) {
      // close: some group that was left out may score as much as one that was kept
      const RouteBounds bd = route_bounds(float(m1), a.group_top2 ? float(m2) : -__builtin_huge_valf(), a.sigmoid);
      const bool kept = (keep >> lane) & 1;
      const float out = wave_max(kept ? -__builtin_huge_valf() : bd.hi);
      const float in = -wave_max(kept ? -bd.lo : -__builtin_huge_valf());
      close = out > -__builtin_huge_valf() && !(out < in);
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const uint32_t g = (uint32_t(lane * KPL + i) * a.group_magic) >> 20;
      if (g >= 64 || !((keep >> g) & 1)) pick[i] = kNone;
    }
    __builtin_amdgcn_wave_barrier();
  }

  // ---- the topk largest picks; one round more shows whether the border was close
  RouteSlot out{-1, 0.f};
  float my_l = -__builtin_huge_valf();
  T my_p = T(0), last = kNone;
  const bool watch = F32 && by_score;
  for (int k = 0; k < a.topk + (watch ? 1 : 0); ++k) {
    T best = pick[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < KPL; ++i)
      if (pick[i] > best) {
        best = pick[i];
        bi = i;
      }
    const T mx = wave_max(best);
    if (!(mx > kNone)) break;
    if constexpr (F32) {
      if (watch && k > 0) close = close || route_near(last, mx, a.sigmoid);
    }
    last = mx;
    if (k == a.topk) break;
    const int win = __builtin_ctzll(__ballot(best == mx));
    float wl = l[0];
    T wp = p[0];
#pragma unroll
    for (int i = 1; i < KPL; ++i)
      if (bi == i) {
        wl = l[i];
        wp = p[i];
      }
    const int id = __builtin_amdgcn_readlane(lane * KPL + bi, win);
    const float ll = lane_value(wl, win);
    const T pp = lane_value(wp, win);
    if (lane == k) {
      out.id = id;
      my_l = ll;
      my_p = pp;
    }
    if (lane == win) {
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (bi == i) pick[i] = kNone;
    }
  }

  // ---- weights
  if (a.renormalize) {
    const float m = wave_max(my_l);
    const T v = out.id >= 0 ? route_ratio<T>(my_l, m, a.sigmoid) : T(0);
    const T tot = wave_total(v);
    out.w = out.id >= 0 ? float(v / tot) * a.scale : 0.f;
  } else {
    out.w = out.id >= 0 ? float(my_p) * a.scale : 0.f;
  }
  return out;
}

}  // namespace mxq
