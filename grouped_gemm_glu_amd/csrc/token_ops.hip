// Launchers of the router, combine and norm kernels.
#include "internal.hpp"
#include "token_ops.hpp"

namespace moe {

namespace {
moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

// workgroups for T tokens whose kernel strides over the rest (a launch stays
// below 2^32 threads)
unsigned token_grid(int T) { return (unsigned)(T < (1 << 20) ? T : (1 << 20)); }

// f(integral_constant<int, VPL>) for the experts per lane of a 64-lane token
template <typename F>
void for_experts_per_lane(int E, F&& f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}
// f(integral_constant<int, NC>) for the 8-column chunks per thread of 256
template <typename F>
void for_chunks(int H, F&& f) {
  if (H <= 2048) f(std::integral_constant<int, 1>{});
  else if (H <= 4096) f(std::integral_constant<int, 2>{});
  else if (H <= 8192) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 8>{});
}
}  // namespace

// Lanes per token of the router: a token takes 16 lanes for up to 256 experts,
// so that four share a wave, unless there are too few tokens to fill two waves
// per SIMD: then a wave each, whose rounds are shorter.  256 experts in 8
// groups, sigmoid and bias, k = 8: 5.0 us with a wave against 7.5 for one token,
// 6.0 / 8.4 for 2048, 7.7 / 8.4 for 4096, 26.4 / 19.4 for 16384; 512 experts (32
// lanes) 4.6 / 6.2, 5.4 / 7.4, 7.3 / 7.2, 21.7 / 17.9; 32 experts 2.9 / 2.8 for one.
int router_lanes(int E, int T) {
  if (E > 64 && T <= 2048) return 64;
  return E <= 256 ? 16 : E <= 512 ? 32 : 64;
}
// f(lanes per token, quads of experts per lane) as integral constants
template <typename F>
void for_router_shape(int E, int lanes, F&& f) {
  using std::integral_constant;
  if (lanes == 16) {
    if (E <= 64) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (E <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    else f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  } else if (lanes == 32) {
    f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  } else if (E <= 256) {
    f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  } else if (E <= 512) {
    f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  } else {
    f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  }
}

moe_status_t launch_router(const RouterArgs& a, bool bf16, int* ids, float* weights, hipStream_t s) {
  if (a.T == 0) return MOE_OK;
  const int lanes = router_lanes(a.E, a.T);
  const int gsz = a.E / a.n_groups;
  const bool fast = a.E % 4 == 0 && (a.n_groups == 1 || (gsz % 4 == 0 && (gsz & (gsz - 1)) == 0 && gsz <= 4 * lanes));
  if (fast) {
    const int per_block = 4 * (64 / lanes);
    const dim3 grid((unsigned)(((long long)a.T + per_block - 1) / per_block));
    for_router_shape(a.E, lanes, [&](auto l, auto n) {
      constexpr int L = decltype(l)::value, NI = decltype(n)::value;
      if (bf16) hipLaunchKernelGGL((router_kernel<L, NI, true>), grid, dim3(256), 0, s, a, ids, weights);
      else hipLaunchKernelGGL((router_kernel<L, NI, false>), grid, dim3(256), 0, s, a, ids, weights);
    });
    return launched();
  }
  const dim3 grid((unsigned)(((long long)a.T + 3) / 4));
  for_experts_per_lane(a.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (bf16) hipLaunchKernelGGL((router_exact_kernel<V, true>), grid, dim3(256), 0, s, a, ids, weights);
    else hipLaunchKernelGGL((router_exact_kernel<V, false>), grid, dim3(256), 0, s, a, ids, weights);
  });
  return launched();
}

moe_status_t launch_router_bwd(const RouterArgs& a, bool bf16, const int* ids, const float* dw,
                               void* dlogits, hipStream_t s) {
  if (a.T == 0) return MOE_OK;
  const dim3 grid((unsigned)(((long long)a.T + 3) / 4));
  for_experts_per_lane(a.E, [&](auto v) {
    if (bf16) hipLaunchKernelGGL((router_bwd_kernel<decltype(v)::value, true>), grid, dim3(256), 0, s, a, ids, dw, dlogits);
    else hipLaunchKernelGGL((router_bwd_kernel<decltype(v)::value, false>), grid, dim3(256), 0, s, a, ids, dw, dlogits);
  });
  return launched();
}

moe_status_t launch_combine(const uint16_t* y, int M_cap, int H, const int* dst, const float* weights,
                            int T, int k, const uint16_t* residual, uint16_t* out, hipStream_t s) {
  if (T == 0) return MOE_OK;
  const dim3 grid(token_grid(T), (unsigned)((H / 8 + 255) / 256));
  hipLaunchKernelGGL(combine_kernel, grid, dim3(256), 0, s, y, M_cap, H, dst, weights, T, k, residual, out);
  return launched();
}

moe_status_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, int M_cap, int H, const int* dst,
                                const float* weights, int T, int k, uint16_t* dy, float* dweights,
                                hipStream_t s) {
  if (T == 0) return MOE_OK;
  hipLaunchKernelGGL(combine_bwd_kernel, dim3(token_grid(T)), dim3(256), 0, s, dout, y, M_cap, H, dst, weights,
                     T, k, dy, dweights);
  return launched();
}

moe_status_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s) {
  if (a.T == 0) return MOE_OK;
  const dim3 grid(token_grid(a.T));
  // few rows: 1024 threads, so that a row is in flight at once (1 row of 7168:
  // 5.6 -> 3.6 us)
  if (a.T <= 512 && a.H > 2048) {
    if (a.H <= 8192) hipLaunchKernelGGL((add_rmsnorm_kernel<1024, 1>), grid, dim3(1024), 0, s, a);
    else hipLaunchKernelGGL((add_rmsnorm_kernel<1024, 2>), grid, dim3(1024), 0, s, a);
  } else {
    for_chunks(a.H, [&](auto nc) {
      hipLaunchKernelGGL((add_rmsnorm_kernel<256, decltype(nc)::value>), grid, dim3(256), 0, s, a);
    });
  }
  return launched();
}

int norm_bwd_parts(int T) { return T < kNormBwdParts ? T : kNormBwdParts; }

moe_status_t launch_add_rmsnorm_bwd(const NormBwdArgs& a, float* dweight, int accumulate, hipStream_t s) {
  const int parts = norm_bwd_parts(a.T);
  if (parts > 0)
    for_chunks(a.H, [&](auto nc) {
      hipLaunchKernelGGL((add_rmsnorm_bwd_kernel<decltype(nc)::value>), dim3((unsigned)parts), dim3(256), 0, s, a);
    });
  if (dweight)
    hipLaunchKernelGGL(norm_dweight_kernel, dim3((unsigned)((a.H + 31) / 32)), dim3(256), 0, s, a.part,
                       parts, a.H, dweight, accumulate);
  return launched();
}

}  // namespace moe
