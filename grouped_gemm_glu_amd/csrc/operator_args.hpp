// Arguments of the router, norm and MXFP4 kernels, shared by the entry points
// and the launchers.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kMaxTopk = 16;
constexpr int kMaxRouterTokens = 1 << 25;   // a launch of 64 lanes per token stays below 2^32
constexpr int kMaxRouterGroups = 64;        // one lane per group
constexpr int kNormMaxH = 16384;
constexpr int kMaxCombineH = 1 << 26;       // 2048 columns per row of the grid
constexpr int kMaxMx4K = 1 << 24;           // a tile's 256 rows of codes, and of outputs, within a
constexpr int kMaxMx4N = 1 << 23;           // descriptor's 2^32 bytes

struct RouterArgs {
  const void* logits;       // fp32 or bf16 [T][E]
  const float* bias;        // [E] or null
  int T, E, k;
  int sigmoid;              // 0: softmax scores
  int n_groups, topk_groups;
  int top2;                 // a group's value: 1 its two best choice values, 0 its best
  int renorm;
  float scale;
};

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;   // or null
  const uint16_t* weight;     // [H]
  int T, H;
  float eps;
  double inv_h;               // 1 / H
  uint16_t* h;                // or null
  uint16_t* y;                // or null
  float* rstd;                // or null
  uint8_t* q;                 // MXFP8 rows of y, or null
  uint8_t* s;
  int e5;
};

struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const uint16_t* weight;
  const float* rstd;
  const uint16_t* dh;         // gradient that reaches h by itself, or null
  int T, H;
  uint16_t* dx;               // or null
  float* part;                // [gridDim.x][H] partial sums of dweight, or null
};

struct Mx4Args {
  const uint8_t* A;         // [M_cap][K/2] e2m1 or [M_cap][K] e4m3 codes
  const uint8_t* a_scales;  // [M_cap][K/32]
  const uint8_t* B;         // [E][N][K/2] e2m1 codes
  const uint8_t* b_scales;  // [E][N][K/32]
  int M_cap, N, K;
  const int* counts;
  int E;
  int* offsets_out;
  int* status_out;
  uint16_t* C;              // [M_cap][N]
};

}  // namespace moe
