// Arguments of the router, norm, MXFP4, adapter and optimizer kernels, shared by
// the entry points and the launchers.
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
constexpr int kMaxLoraRank = 128;
constexpr int kMaxLoraRows = 1 << 25;       // a launch of 256 threads per 16 rows stays below 2^32
constexpr int kMaxLoraCols = 1 << 17;       // 1024 of r times as many per row of the grid

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

// Rows of adapters: group e's are grouped rows o_e .. o_e + counts[e].
struct LoraGroups {
  const int* counts;        // [L]
  int L, M_cap;
  int* offsets_out;
  int* status_out;
  const int* src;           // [M_cap]: grouped row -> row of x and y, or null: the same
  int T;                    // rows of x and y
};

struct LoraArgs {
  LoraGroups g;
  const uint16_t* A;        // [L][r][K]
  const uint16_t* B;        // [L][N][r]
  const float* scale;       // [L] or null
  int r, K, N;
  long long x_ld, y_ld;
};

// A piece of a tensor of an AdamW step, as the device's table holds it: everything
// that its workgroup needs, so that one load leads to the elements.
struct AdamwChunk {
  void* param;              // its first element; null: the tensor takes part in the norm alone
  const void* grad;
  float* master;            // null: the parameter is its own
  void* m;
  void* v;
  float* m_scale;           // 8-bit states: one of each per kAdamwBlock elements
  float* v_scale;
  float lr_scale, decay;
  int n;                    // elements
  uint16_t param_bf16, grad_bf16;
};
constexpr int kAdamwBlock = 128;
constexpr int kAdamwStep = 1024;            // elements of a workgroup's step; a chunk is 2 or 4 of them
constexpr int kNormParts = 1024;            // workgroups, at most, of the gradients' norm

struct AdamwArgs {
  const AdamwChunk* chunks;
  long long n_chunks, n_chunks8;   // all, those of 8-bit states (the last ones)
  double lr, beta1, beta2, eps;
  double bias1, bias2;      // 1 - beta^step, where the step is not the device's
  const int* step;          // device, or null
  const float* lr_dev;      // device, or null
  const float* grad_scale;  // device, or null
};

}  // namespace moe
