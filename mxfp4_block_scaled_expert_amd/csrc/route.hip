// Expert routing: router logits [M, E] -> expert ids and weights [M, topk] (route_common.hpp holds
// the formulas).  One wave per token, four tokens per workgroup.  Scores are computed in fp32;
// where two picks that decide the result lie closer than fp32 scores can tell apart, the wave
// repeats its token in 64 bits, so the chosen experts and their order are those of the exact
// scores.
#include "kernels.hpp"
#include "route_common.hpp"

namespace mxq {

namespace {
constexpr int kRouteWaves = 4;
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

void launch_moe_route(const void* logits, bool bf16, int64_t M, int64_t ld, const RouteArgs& a, int32_t* ids,
                      float* weights, hipStream_t stream) {
  if (M <= 0) return;
  const dim3 grid{unsigned(cdiv(M, kRouteWaves))}, block{256u};
  const size_t lds = a.n_group > 1 ? size_t(kRouteWaves) * a.E * 8 : 0;
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
