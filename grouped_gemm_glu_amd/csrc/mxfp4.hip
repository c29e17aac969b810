// Launchers of the MXFP4 quantisation and grouped product.
#include <algorithm>
#include <cmath>

#include "internal.hpp"
#include "mxfp4.hpp"

namespace moe {

namespace {
moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

// Whether M rows in E groups go to the kernel that streams the weights past 16
// rows of a group at a time, or to the 256 x 256 tiles: the smaller of two
// estimates in microseconds, whose constants are measured (4-bit / 8-bit rows).  M
// is the capacity: how many rows there are, and in how many groups, is on the
// device alone.
//   rows:  the weights of the groups that can be there, or of all 16-row tiles,
//          at 5.0 / 4.3 TB/s, and up to 40% more as 16 rows are reached
//   tiles: 1.5 / 2.4 us per 256 values of K and round of tiles over the compute
//          units, or the weights at 4.2 / 3.35 TB/s
// E = 32, N = 4096, K = 7168, 4-bit rows: 1 row per group 100 us against 118 with
// tiles, 4 rows 108 / 120, 8 rows 118 / 117, 16 rows 138 / 118, 32 rows 233 / 122;
// E = 1, N = 2048, K = 7168, 8 rows: 7 against 33.
bool few_rows(int M_cap, int E, int N, int K, bool a4, int cus) {
  const double M = M_cap, w = (double)N * K * (0.5 + 1.0 / 32) * 1e-6;   // MB of a group's weights
  const double act = std::min<double>(E, M), per = std::min(16.0, M / act);
  const double part = std::min(1.0, cus / 128.0);   // about half the units reach the memory's rate
  const double rows = std::max(act, M / 16) * w / (a4 ? 5.0 : 4.3) / part * (1 + per / 40) + 4;
  const double rounds = std::ceil(std::max(act, M / MX4_BM) * ((N + MX4_BN - 1) / MX4_BN) / cus);
  const double tiles = std::max(rounds * ((K + 255) / 256) * (a4 ? 1.5 : 2.4), act * w / (a4 ? 4.2 : 3.35) / part) + 6;
  return rows < tiles;
}

}  // namespace

// (the tiles load 16 scales at once, which their arrays have to hold)
extern "C" int moe_mx4_takes_tiles(int M_cap, int E, int N, int K, int a4, int cus) {
  return (long long)M_cap * (K / 32) >= 16 && !few_rows(M_cap, E, N, K, a4 != 0, cus);
}

moe_status_t launch_mx4_rows(const uint16_t* v, int R, int C, const int* counts, int E, uint8_t* q,
                             uint8_t* s, int cus, hipStream_t st) {
  const long long chunks = (long long)R * (C / 8);
  if (chunks == 0) return MOE_OK;
  // four chunks in flight per thread where that still fills the chip
  if (chunks >= (long long)cus * 8 * 1024) {
    hipLaunchKernelGGL(mx4_rows_kernel<4>, dim3(cus * 8), dim3(256), 0, st, v, R, C, counts, E, q, s);
  } else {
    const int grid = (int)std::min<long long>((chunks + 255) / 256, cus * 8LL);
    hipLaunchKernelGGL(mx4_rows_kernel<1>, dim3(grid), dim3(256), 0, st, v, R, C, counts, E, q, s);
  }
  return launched();
}

moe_status_t launch_mx4_weight_kn(const uint16_t* src, int E, int N, int K, uint8_t* q, uint8_t* s,
                                  hipStream_t st) {
  hipLaunchKernelGGL(mx4_weight_kn_kernel, dim3((N + 255) / 256, K / 32, E), dim3(256), 0, st, src, N, K, q, s);
  return launched();
}

moe_status_t launch_mx4_gemm(const Mx4Args& a, bool a4, int cus, hipStream_t st) {
  if (a.M_cap == 0 && !a.offsets_out && !a.status_out) return MOE_OK;
  if (moe_mx4_takes_tiles(a.M_cap, a.E, a.N, a.K, a4, cus)) {
    const long long tiles = ((long long)(a.M_cap + MX4_BM - 1) / MX4_BM + a.E) * ((a.N + MX4_BN - 1) / MX4_BN);
    const int g = (int)std::min<long long>(tiles, cus);
    if (a4) hipLaunchKernelGGL(mx4_gemm_tile_kernel<true>, dim3(g), dim3(512), 0, st, a);
    else hipLaunchKernelGGL(mx4_gemm_tile_kernel<false>, dim3(g), dim3(512), 0, st, a);
    return launched();
  }
  // the most tiles of 16 rows that M_cap rows in E groups can make
  const long long tiles = std::min<long long>((a.M_cap + 15LL) / 16 + a.E, a.M_cap);
  // K split over a workgroup's waves where there are fewer items of 64 columns
  // than half the compute units: E = 1, N = 2048, K = 7168, 8 rows 7.4 us against
  // 16.3 whole; 4 groups of N = K = 2880 (180 items) 8.2 against 7.9
  const bool split = 2 * tiles * (a.N / 64) < cus;
  const long long items = tiles * (split ? a.N / 16 : a.N / 64);
  const int g = (int)std::max(1LL, std::min<long long>(items, cus * 8LL));   // (without rows: offsets and status)
  auto go = [&](auto a4c, auto se, auto sp) {
    hipLaunchKernelGGL((mx4_gemm_rows_kernel<decltype(a4c)::value, decltype(se)::value, decltype(sp)::value>),
                       dim3(g), dim3(256), 0, st, a);
  };
  auto go2 = [&](auto a4c, auto se) {
    if (split) go(a4c, se, std::true_type{});
    else go(a4c, se, std::false_type{});
  };
  auto go1 = [&](auto a4c) {
    if (a.E <= 64) go2(a4c, std::true_type{});
    else go2(a4c, std::false_type{});
  };
  if (a4) go1(std::true_type{});
  else go1(std::false_type{});
  return launched();
}

}  // namespace moe
