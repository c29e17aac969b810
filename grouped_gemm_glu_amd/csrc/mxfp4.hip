// Launchers of the MXFP4 quantisation and grouped product.
#include "internal.hpp"
#include "mxfp4.hpp"

namespace moe {

namespace {
moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }
}  // namespace

moe_status_t launch_mx4_rows(const uint16_t* v, int R, int C, const int* counts, int E, uint8_t* q,
                             uint8_t* s, int cus, hipStream_t st) {
  const long long blocks = ((long long)R * (C / 8) + 255) / 256;
  if (blocks == 0) return MOE_OK;
  const int grid = (int)(blocks < (long long)cus * 8 ? blocks : (long long)cus * 8);
  hipLaunchKernelGGL(mx4_rows_kernel, dim3(grid), dim3(256), 0, st, v, R, C, counts, E, q, s);
  return launched();
}

moe_status_t launch_mx4_weight_kn(const uint16_t* src, int E, int N, int K, uint8_t* q, uint8_t* s,
                                  hipStream_t st) {
  hipLaunchKernelGGL(mx4_weight_kn_kernel, dim3((N + 255) / 256, K / 32, E), dim3(256), 0, st, src, N, K, q, s);
  return launched();
}

moe_status_t launch_mx4_gemm(const Mx4Args& a, bool a4, int cus, hipStream_t st) {
  if (a.M_cap > 32LL * a.E && a.K >= 256) {
    const long long tiles = ((long long)(a.M_cap + MX4_BM - 1) / MX4_BM + a.E) * ((a.N + MX4_BN - 1) / MX4_BN);
    const int g = (int)(tiles < cus ? tiles : cus);
    if (a4) hipLaunchKernelGGL(mx4_gemm_tile_kernel<true>, dim3(g), dim3(512), 0, st, a);
    else hipLaunchKernelGGL(mx4_gemm_tile_kernel<false>, dim3(g), dim3(512), 0, st, a);
    return launched();
  }
  const long long items = ((long long)(a.M_cap + 63) / 64 + a.E) * (a.N / 16);
  const int grid = (int)(items < (long long)cus * 8 ? items : (long long)cus * 8);
  if (a4) hipLaunchKernelGGL((mx4_gemm_small_kernel<true, 4>), dim3(grid), dim3(256), 0, st, a);
  else hipLaunchKernelGGL((mx4_gemm_small_kernel<false, 4>), dim3(grid), dim3(256), 0, st, a);
  return launched();
}

}  // namespace moe
