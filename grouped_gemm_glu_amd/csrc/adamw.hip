// Launchers of the AdamW and gradient norm kernels.
#include "internal.hpp"
#include "adamw.hpp"

namespace moe {

namespace {
moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }
}  // namespace

moe_status_t launch_adamw(const AdamwArgs& a, int cus, hipStream_t s) {
  if (a.n_chunks == 0) return MOE_OK;
  const long long most = 8LL * cus;
  hipLaunchKernelGGL(adamw_kernel, dim3((unsigned)(a.n_chunks < most ? a.n_chunks : most)), dim3(256), 0, s, a);
  return launched();
}

moe_status_t launch_adamw_unpack(const int8_t* m, const float* m_scale, const uint8_t* v, const float* v_scale,
                                 long long n, float* m_out, float* v_out, hipStream_t s) {
  if (n == 0) return MOE_OK;
  const long long blocks = (n + 1023) / 1024;
  hipLaunchKernelGGL(adamw_unpack_kernel, dim3((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20))), dim3(256), 0, s, m,
                     m_scale, v, v_scale, n, m_out, v_out);
  return launched();
}

moe_status_t launch_grad_norm(const AdamwTensor* tensors, const AdamwChunk* chunks, long long n_chunks, float max_norm,
                              float* out, double* part, hipStream_t s) {
  const int parts = (int)(n_chunks < kNormParts ? n_chunks : kNormParts);
  if (parts > 0)
    hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)parts), dim3(256), 0, s, tensors, chunks, n_chunks, part);
  hipLaunchKernelGGL(grad_norm_final_kernel, dim3(1), dim3(256), 0, s, part, parts, max_norm, out);
  return launched();
}

}  // namespace moe
