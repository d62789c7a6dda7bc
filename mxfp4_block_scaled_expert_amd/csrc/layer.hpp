// Launchers and argument structures of expert routing, the few-token MoE layer and the 4-bit linear.
#pragma once

#include "kernels.hpp"

namespace mxq {

constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxTopk = 32;
constexpr int kRouteMaxGroups = 64;

// How a token's experts are chosen (route_common.hpp).
struct RouteArgs {
  int32_t E, topk;
  int32_t sigmoid;          // 1: sigmoid scores, 0: softmax
  int32_t n_group, topk_group;
  int32_t group_top2;       // group score: 1 the two largest p + bias, 0 the largest pick
  int32_t renormalize;
  float scale;
  const float* bias;        // [E] correction bias or NULL
  int32_t group_size;       // E / n_group
  uint32_t group_magic;     // ceil(2^20 / group_size): e / group_size = (e * magic) >> 20 for e < 512
};
// logits fp32 or bf16 [M, E] (row stride ld elements) -> ids int32 [M, topk], weights fp32 [M, topk]
void launch_moe_route(const void* logits, bool bf16, int64_t M, int64_t ld, const RouteArgs& a, int32_t* ids,
                      float* weights, hipStream_t stream);

// A whole routed-expert layer for at most kLayerMaxTokens tokens (moe_layer.hip).
constexpr int kLayerMaxTokens = 16;
struct LayerArgs {
  const uint16_t* x;        // bf16 [M_all, H], row stride ldx elements
  int64_t ldx, H, I;
  int32_t M_all;            // tokens of the call
  int32_t t0, M;            // tokens of this pass: [t0, t0 + M)
  const void* gate;         // [E, H] bf16 or fp32
  int32_t gate_f32;
  const float* gate_bias;   // [E] or NULL
  RouteArgs rt;
  int32_t wfmt;             // W_E4M3_BLOCK or W_E2M1_MX
  int32_t tiled;
  const uint8_t *w1, *s1, *w2, *s2;
  const float* b1;          // [E, 2I] or NULL
  float* part;              // [S][M_all][E] partial logits
  int32_t S, chunk;         // K chunks of the router product
  uint16_t* h;              // [sorted row][hi, lo][I] bf16
  int32_t* rows;            // the pass's routing for the down stage, R = M * topk: row count | [R] sorted
                            // rows (expert << 8 | token) | [R] sorted row of flat row t * topk + k or -1
                            // | [E] tokens of each expert, one bit per token
  uint16_t* out;            // bf16 [M_all, H], row stride ldo elements
  int64_t ldo;
};
// Tokens one pass of the expert stages can take (their rows of x, and the sums of their rows, lie in LDS), and the K chunks of
// the router product.
int layer_pass_tokens(int wfmt, int64_t H, int32_t E, int32_t topk);
void layer_gate_split(int32_t E, int64_t H, int32_t& S, int32_t& chunk);
void launch_moe_layer(const LayerArgs& a, hipStream_t stream);

// Linear with 4-bit weights and group scales (int4.hip).
struct Int4Args {
  const void* A;            // bf16 [M, K], row stride lda elements
  int64_t lda;
  const uint8_t* W;         // [N, K/2], element 2j in the low nibble of byte j
  const void* s;            // [N, K/G] fp32 or bf16
  int32_t s_bf16;
  const uint8_t* z;         // [N, ceil(K/G/2)] zero points, group 2j in the low nibble; NULL: 8
  const void* bias;         // [N] fp32 or bf16, or NULL
  int32_t bias_bf16;
  void* out;                // bf16 [M, N], row stride ldo; K split: fp32 [splits][M][N]
  int64_t ldo;
  int64_t M, N, K;
  int32_t group;
  int32_t splits, split_steps;  // K chunks of split_steps 128-wide steps
  int64_t split_stride;
};
struct Int4Plan {
  int32_t mt;               // 16-row tiles per workgroup; 0: the dot-product kernel
  int32_t splits, split_steps;
  size_t partial_bytes;
};
Int4Plan int4_plan(int64_t M, int64_t N, int64_t K, int group);
// group 32, 64 or 128; `partial`: int4_plan's partial_bytes of workspace
void launch_int4_linear(const Int4Args& a, int group, float* partial, hipStream_t stream);

}  // namespace mxq
