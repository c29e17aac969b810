// Launchers of the AdamW and gradient norm kernels.
#include "internal.hpp"
#include "adamw.hpp"

namespace moe {

namespace {
moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }
}  // namespace

moe_status_t launch_adamw(const AdamwArgs& a, int cus, hipStream_t s) {
  const long long n32 = a.n_chunks - a.n_chunks8;
  // Workgroups per compute unit, striding over the rest.  32 bits: 5 to 8 streams,
  // which more workgroups scatter over memory (531M elements: 2 3.18 ms, 3 3.13, 4
  // 3.21; 3 is 5.1 TB/s); 8 bits: its 64-bit arithmetic wants the waves (265M: 4 1.34
  // ms, 8 0.99, 4.9 TB/s).
  const auto grid = [&](long long n, int per_cu) {
    const long long most = (long long)per_cu * cus;
    return dim3((unsigned)(n < most ? n : most));
  };
  if (n32 > 0)
    hipLaunchKernelGGL(adamw_kernel<false>, grid(n32, 3), dim3(256), 0, s, a, a.chunks, 0LL, n32);
  if (a.n_chunks8 > 0)
    hipLaunchKernelGGL(adamw_kernel<true>, grid(a.n_chunks8, 8), dim3(256), 0, s, a, a.chunks, n32, a.n_chunks);
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

moe_status_t launch_grad_norm(const AdamwChunk* chunks, long long n_chunks, float max_norm, float* out, double* part,
                              hipStream_t s) {
  // One workgroup for few chunks (us against two launches: 16 chunks of 2048 4.0 / 6.9, 32 5.5 /
  // 7.0, 48 7.4 / 7.0, 64 9.1 / 6.9).
  if (n_chunks <= 32) {
    hipLaunchKernelGGL(grad_norm_few_kernel, dim3(1), dim3(1024), 0, s, chunks, n_chunks, max_norm, out);
    return launched();
  }
  // (265M fp32 gradients: 1024 workgroups 165 us, 6.4 TB/s; 768 the same, 512 218)
  const int parts = (int)(n_chunks < kNormParts ? n_chunks : kNormParts);
  hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)parts), dim3(256), 0, s, chunks, n_chunks, part);
  hipLaunchKernelGGL(grad_norm_final_kernel, dim3(1), dim3(256), 0, s, part, parts, max_norm, out);
  return launched();
}

}  // namespace moe
