// Host-side declarations shared by the library's translation units.
#pragma once

#include <hip/hip_runtime.h>

#include "group_gemm.hpp"
#include "moe_glu.h"
#include "operator_args.hpp"

namespace moe {

// Launch one persistent grouped-GEMM kernel instantiation; each returns
// MOE_ERR_UNSUPPORTED for a combination its translation unit does not hold.
moe_status_t launch_group_gemm_fwd(int epi, int blay, const GemmArgs& args, int grid,
                                   hipStream_t stream);
moe_status_t launch_group_gemm_bwd(int epi, int blay, const GemmArgs& args, int grid,
                                   hipStream_t stream);
// MXFP8 x MXFP8 GroupGemm (packed MXFP8 weight, bf16 output); a_e5: A holds
// e5m2 codes
moe_status_t launch_group_gemm_mx(const GemmArgs& args, bool a_e5, int grid, hipStream_t stream);

// Kernels whose epilogue applies the activation exist once per activation
// (gemm_act_fwd.hip and gemm_act_bwd.hip are compiled once per value of
// MOE_ACT); launch_activation_kernel picks the one for args.ep.act.
enum {
  KIND_GLU = 0,          // FC1 + GLU, bf16 operands, packed W1
  KIND_GLU_MXO,          // the same with MXFP8 outputs
  KIND_MXIN_GLU,         // FC1 + GLU, MXFP8 operands
  KIND_MXIN_GLU_MXO,     // the same with MXFP8 outputs
  KIND_ACT,              // FC1 + non-gated activation, packed plain W1
  KIND_DGLU_PACKED,      // dgrad + dGLU, packed W2 (this and the kinds below: backward)
  KIND_DGLU_NK,          // dgrad + dGLU, W2 as [I][H]
  KIND_DGLU_G_PACKED,    // the same two adding d(bias) and d(row_scale)
  KIND_DGLU_G_NK,
  KIND_DACT_PACKED,      // dgrad + non-gated activation derivative
  KIND_DACT_NK
};
moe_status_t launch_activation_kernel(int kind, const GemmArgs& args, int grid, hipStream_t stream);
#define MOE_DECLARE_ACT_LAUNCHERS(n)                                                              \
  moe_status_t launch_act_fwd_##n(int kind, const GemmArgs& args, int grid, hipStream_t stream); \
  moe_status_t launch_act_bwd_##n(int kind, const GemmArgs& args, int grid, hipStream_t stream);
MOE_DECLARE_ACT_LAUNCHERS(0)
MOE_DECLARE_ACT_LAUNCHERS(1)
MOE_DECLARE_ACT_LAUNCHERS(2)
MOE_DECLARE_ACT_LAUNCHERS(3)
#undef MOE_DECLARE_ACT_LAUNCHERS
// K-grouped weight gradient (fp32 output)
moe_status_t launch_group_gemm_wgrad(const GemmArgs& args, int grid, hipStream_t stream);
// the same on K-tiled MXFP8 column copies; a_e5 / b_e5: e5m2 codes
moe_status_t launch_group_gemm_wgrad_mx(const GemmArgs& args, bool a_e5, bool b_e5, int grid,
                                        hipStream_t stream);

// Router, combine and norm (token_ops.hip); T = 0 launches nothing
moe_status_t launch_router(const RouterArgs& a, bool bf16, int* ids, float* weights, hipStream_t s);
moe_status_t launch_router_bwd(const RouterArgs& a, bool bf16, const int* ids, const float* dw,
                               void* dlogits, hipStream_t s);
moe_status_t launch_combine(const uint16_t* y, int M_cap, int H, const int* dst, const float* weights,
                            int T, int k, const uint16_t* residual, uint16_t* out, hipStream_t s);
moe_status_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, int M_cap, int H, const int* dst,
                                const float* weights, int T, int k, uint16_t* dy, float* dweights,
                                hipStream_t s);
moe_status_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s);
// rows of partial dweight sums that the backward writes (its workgroups)
constexpr int kNormBwdParts = 512;
int norm_bwd_parts(int T);
moe_status_t launch_add_rmsnorm_bwd(const NormBwdArgs& a, float* dweight, int accumulate, hipStream_t s);

// Low-rank adapters (lora.hip).  The sizes of a call, from which its launches and
// its workspace follow; the same for every device.
struct LoraShape {
  int M_cap, L, r, K, N;
};
size_t lora_fwd_workspace(const LoraShape& s);
size_t lora_bwd_workspace(const LoraShape& s);
// Which kernels a call of these sizes takes: out[0] for u and y, out[1] for w and
// dx (0 one launch, 1 two of 16-row tiles, 2 and 3 two of tiles of 64 and of 128
// rows), out[2] the most rows of a piece of dA and dB.  Not part of the public
// interface; a symbol of its own so that a test of a kernel can tell that its
// sizes reach it.
extern "C" void moe_lora_takes(int M_cap, int E, int r, int K, int N, int* out);
moe_status_t launch_lora_fwd(const LoraArgs& a, const uint16_t* x, const uint16_t* base, uint16_t* y, float* u,
                             void* ws, hipStream_t s);
moe_status_t launch_lora_bwd(const LoraArgs& a, const uint16_t* dy, const uint16_t* x, const float* u,
                             const uint16_t* dx_base, uint16_t* dx, float* dA, float* dB, int accumulate, void* ws,
                             hipStream_t s);

// AdamW and the gradients' norm (adamw.hip)
moe_status_t launch_adamw(const AdamwArgs& a, int cus, hipStream_t s);
moe_status_t launch_adamw_unpack(const int8_t* m, const float* m_scale, const uint8_t* v, const float* v_scale,
                                 long long n, float* m_out, float* v_out, hipStream_t s);
moe_status_t launch_grad_norm(const AdamwChunk* chunks, long long n_chunks, float max_norm, float* out, double* part,
                              hipStream_t s);

// MXFP4 (mxfp4.hip); a4: e2m1 rows, else e4m3
moe_status_t launch_mx4_rows(const uint16_t* v, int R, int C, const int* counts, int E, uint8_t* q,
                             uint8_t* s, int cus, hipStream_t st);
moe_status_t launch_mx4_weight_kn(const uint16_t* src, int E, int N, int K, uint8_t* q, uint8_t* s,
                                  hipStream_t st);
moe_status_t launch_mx4_gemm(const Mx4Args& a, bool a4, int cus, hipStream_t st);
// Whether such a product of cus compute units goes to the 256 x 256 tiles, or to
// the kernel that streams the weights past 16 rows at a time.  Not part of the
// public interface; a symbol of its own so that a test of a kernel can tell that
// its sizes reach it.
extern "C" int moe_mx4_takes_tiles(int M_cap, int E, int N, int K, int a4, int cus);

}  // namespace moe
