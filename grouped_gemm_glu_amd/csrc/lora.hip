// Launchers of the adapter kernels.
#include <algorithm>

#include "internal.hpp"
#include "lora.hpp"

namespace moe {

namespace {
moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }
int div_up(long long a, long long b) { return (int)((a + b - 1) / b); }
size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

// An upper bound of the tiles (each group adds at most one partial tile), and
// what to expect when groups end in the middle of one.
unsigned tile_bound(int M_cap, int L, int bm) { return (unsigned)(M_cap / bm + (L < M_cap ? L : M_cap)); }
int tile_guess(int M_cap, int L, int bm) { return M_cap / bm + (L < M_cap ? L : M_cap) / 2; }
// 16-row blocks per wave: two where groups fill them (fewer reads of the weights)
int narrow_blocks(const LoraShape& s) { return s.M_cap < 128LL * s.L ? 1 : 2; }
// Columns per workgroup, a multiple of 128, for about `target` workgroups.
int slice_of(int cols, int tiles, int target) {
  const int n = target / (tiles > 0 ? tiles : 1);
  return div_up(div_up(cols, n > 0 ? n : 1), 128) * 128;
}
// About 640 workgroups, in 8 slices at most, which every workgroup of the wide kernel adds
// up (us of the two kernels, N 4096: 256 rows, r 64, K 7168: 56 slices 6.9 + 21.2, 24 6.8 +
// 12.7, 8 11.4 + 9.8; 4096 rows, r 8, K 7168: 19 slices 20.2 + 19.5, 8 20.2 + 16.6; 2048 rows,
// r 64, K and N 2880: 23 slices 9.5 + 18.6, 8 10.1 + 15.4).
int narrow_slice(const LoraShape& s, int K) {
  const int most = div_up(div_up(K, 8), 128) * 128;
  return std::max(most, slice_of(K, tile_guess(s.M_cap, s.L, 64 * narrow_blocks(s)), 640));
}
// About 832 workgroups (512 of the larger LDS of r > 64), of three steps at least where
// there are tiles enough (2048 rows in 64 groups, r 16, N 2880: slices of 128 columns 12.7
// us, 384 10.2, 512 11.3; 256 rows, r 64, N 4096: 9.8, 12.3, 14.2; 16384 rows, r 64, N 4096:
// 3 slices 53.8, 2 61.5, 4 64.7).
int wide_slice(const LoraShape& s, int N) {
  const int tiles = tile_guess(s.M_cap, s.L, 64);
  return std::max(tiles < 32 ? 128 : 384, slice_of(N, tiles, s.r > 64 ? 512 : 832));
}
size_t partial_bytes(const LoraShape& s, int K) {
  return aligned((size_t)div_up(K, narrow_slice(s, K)) * (size_t)s.M_cap * (size_t)s.r * 4);
}
int sum_blocks(int r, int C) { return div_up(C, r <= 64 ? 512 : 256); }
// Rows per workgroup of the sums, a multiple of 64, for about 448 workgroups beside the
// groups' last pieces; two or three run on a compute unit (16384 rows, K 7168, N 4096, 32
// groups of r 32: 320 142 us, 448 127, 512 130; 8 groups of r 64: 122, 120, 142).
int sum_piece(const LoraShape& s) {
  const long long p = (long long)s.M_cap * (sum_blocks(s.r, s.K) + sum_blocks(s.r, s.N)) / 448;
  return p <= 128 ? 128 : p >= kLoraPiece ? kLoraPiece : div_up(p, 64) * 64;
}
// Groups of more rows than a piece, at most, and their pieces: ceil(m / p) <= m / p + 1.
int many_groups(const LoraShape& s) {
  const int n = s.M_cap / (sum_piece(s) + 1);
  return n < s.L ? n : s.L;
}
size_t sum_slots(const LoraShape& s) { return (size_t)(s.M_cap / sum_piece(s)) + (size_t)many_groups(s); }
// Whether one launch does both products of the forward: every workgroup of a tile
// reads the whole A, which pays while that is short beside a launch (3.2 us on the
// host) and the tiles leave more than one workgroup for few compute units alone; the LDS
// of a larger r holds one or two workgroups on each.  Us of two launches against one, N
// 4096: 1 row, r 16: K 2880 9.5 / 5.9, K 7168 9.3 / 7.7, K 16384 9.6 / 13.0; r 32, K 4096 9.6
// / 7.8; r 64, K 2048 10.3 / 9.2; 64 rows in 32 groups, r 128, K 1024 29.2 / 21.8; 1024 rows
// in 4 groups (68 tiles): r 16, K 7168 18.0 / 13.3; r 64, K 2048 21.8 / 21.1; r 128, K 1024
// 29.1 / 33.5; 3000 rows in 8 groups (195): r 16, K 2880 20.0 / 17.4; r 32 24.1 / 23.3; r 64,
// K 1024 28.1 / 40.0; 4096 rows (264), r 16, K 2880 23.3 / 27.3.
bool fused_rows(const LoraShape& s) {
  const unsigned most = s.r <= 32 ? 256 : s.r <= 64 ? 128 : 64;
  return s.r * s.K <= (1 << 17) && tile_bound(s.M_cap, s.L, 16) <= most;
}
// The same for the backward's w and dx, whose weights of r > 32 do not fit the LDS.  Us of a
// forward and a backward, w and dx in two launches against one, K 4096: 16 rows, r 16, N 1024
// 18.1 / 15.7; 100 rows in 4 groups, r 32, N 1024 25.7 / 21.9; 1024 rows, r 16, N 2880 35.8 /
// 32.1; 1500 rows in 96 groups (189 tiles), r 16, N 1024 65.3 / 54.6; 2000 rows in 8 groups
// (133), r 32, N 1024 48.9 / 47.2, N 4096 72.4 / 74.7; 3000 rows in 8 groups (195), r 16, N
// 2880 62.8 / 62.5, r 32, N 1024 58.4 / 54.9, N 4096 86.7 / 87.8: no more to gain where both
// are near their end, 1 to 3% lost.
bool fused_back(const LoraShape& s) {
  return s.r <= 32 && s.r * s.N <= (1 << 17) && tile_bound(s.M_cap, s.L, 16) <= 256;
}
// Else, whether it goes by tiles of 16 rows (2048 rows in 64 groups, r 16, K and N 2880: 30.5
// us, with tiles of 64 rows 22.3).
bool few_rows(const LoraShape& s) { return s.M_cap <= 64 || s.M_cap <= 4LL * s.L; }

template <typename F>
void for_rank_blocks(int r, F&& f) {
  if (r <= 16) f(std::integral_constant<int, 1>{});
  else if (r <= 32) f(std::integral_constant<int, 2>{});
  else if (r <= 64) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 8>{});
}

struct BwdLayout {
  size_t w, narrow, sumA, sumB, end;
};
BwdLayout bwd_layout(const LoraShape& s) {
  BwdLayout l;
  l.w = 0;
  l.narrow = aligned((size_t)s.M_cap * s.r * 4);
  l.sumA = l.narrow + partial_bytes(s, s.N);
  l.sumB = l.sumA + aligned(sum_slots(s) * (size_t)s.r * s.K * 4);
  l.end = l.sumB + aligned(sum_slots(s) * (size_t)s.r * s.N * 4);
  return l;
}

template <bool TURNED>
void narrow(const LoraGroups& g, const LoraShape& s, const uint16_t* x, long long x_ld, const uint16_t* W, int K,
            int slice, float* out, hipStream_t st) {
  const int mb = narrow_blocks(s);
  const dim3 grid(tile_bound(s.M_cap, s.L, 64 * mb), (unsigned)div_up(K, slice));
  for_rank_blocks(s.r, [&](auto n) {
    constexpr int RB = decltype(n)::value;
    if (mb == 1)
      hipLaunchKernelGGL((lora_narrow_kernel<RB, 1, TURNED>), grid, dim3(256), 0, st, g, x, x_ld, W, s.r, K, slice, out);
    else
      hipLaunchKernelGGL((lora_narrow_kernel<RB, 2, TURNED>), grid, dim3(256), 0, st, g, x, x_ld, W, s.r, K, slice, out);
  });
}

template <bool TURNED>
void wide(const LoraGroups& g, const LoraShape& s, const float* u, int slices, float* u_out, const uint16_t* W, int N,
          const float* scale, const uint16_t* base, uint16_t* y, long long y_ld, hipStream_t st) {
  const int slice = wide_slice(s, N);
  const dim3 grid(tile_bound(s.M_cap, s.L, 64), (unsigned)div_up(N, slice));
  for_rank_blocks(s.r, [&](auto n) {
    hipLaunchKernelGGL((lora_wide_kernel<decltype(n)::value, TURNED>), grid, dim3(256), 0, st, g, u, slices, u_out, W,
                       scale, s.r, N, slice, base, y, y_ld);
  });
}

// Both products in one launch: W1 has K columns, W2 N.
template <bool TURNED>
void few(const LoraGroups& g, const LoraShape& s, const uint16_t* x, long long x_ld, const uint16_t* W1, const uint16_t* W2,
         int K, int N, const float* scale, const uint16_t* base, uint16_t* y, long long y_ld, float* u, hipStream_t st) {
  const unsigned tiles = tile_bound(s.M_cap, s.L, 16);
  // columns for 256 workgroups (512: 64 rows in 32 groups 9.4 us for 7.4); where there are
  // more than eight waves take at once, they take two runs at a time
  const int slice = div_up(div_up(N, (int)(256 / tiles)), 256) * 256;
  const dim3 grid(tiles, (unsigned)div_up(N, slice));
  const auto go = [&](auto rb, auto nb) {
    constexpr int RB = decltype(rb)::value, NB = decltype(nb)::value;
    hipLaunchKernelGGL((lora_few_kernel<RB, RB <= 2 ? 2 : 1, NB, TURNED>), grid, dim3(512), 0, st, g, x, x_ld, W1, W2, scale,
                       s.r, K, N, slice, base, y, y_ld, u);
  };
  for_rank_blocks(s.r, [&](auto n) {
    if constexpr (decltype(n)::value <= 2) {
      if (slice > 256) return go(n, std::integral_constant<int, 2>{});
    }
    if constexpr (decltype(n)::value <= 2 || !TURNED) go(n, std::integral_constant<int, 1>{});
  });
}

moe_status_t report(const LoraGroups& g, hipStream_t st) {
  if (g.offsets_out || g.status_out) hipLaunchKernelGGL(lora_report_kernel, dim3(1), dim3(64), 0, st, g);
  return launched();
}
}  // namespace

size_t lora_fwd_workspace(const LoraShape& s) {
  if (fused_rows(s)) return 0;
  return few_rows(s) ? aligned((size_t)div_up(s.K, 512) * (size_t)s.M_cap * (size_t)s.r * 4) : partial_bytes(s, s.K);
}
size_t lora_bwd_workspace(const LoraShape& s) { return bwd_layout(s).end; }

extern "C" void moe_lora_takes(int M_cap, int E, int r, int K, int N, int* out) {
  const LoraShape s = {M_cap, E, r, K, N};
  out[0] = fused_rows(s) ? 0 : few_rows(s) ? 1 : 1 + narrow_blocks(s);
  out[1] = fused_back(s) ? 0 : 1 + narrow_blocks(s);
  out[2] = sum_piece(s);
}

moe_status_t launch_lora_fwd(const LoraArgs& a, const uint16_t* x, const uint16_t* base, uint16_t* y, float* u,
                             void* ws, hipStream_t st) {
  const LoraShape s = {a.g.M_cap, a.g.L, a.r, a.K, a.N};
  if (a.g.M_cap == 0 || a.g.T == 0) return report(a.g, st);
  if (fused_rows(s)) {
    few<false>(a.g, s, x, a.x_ld, a.A, a.B, a.K, a.N, a.scale, base, y, a.y_ld, u, st);
    return launched();
  }
  const unsigned tiles = tile_bound(s.M_cap, s.L, 16);
  if (few_rows(s)) {
    const int slices = div_up(a.K, 512);
    float* part = slices == 1 && u ? u : static_cast<float*>(ws);
    for_rank_blocks(s.r, [&](auto n) {
      constexpr int RB = decltype(n)::value;
      hipLaunchKernelGGL((lora_few_narrow_kernel<RB>), dim3(tiles, (unsigned)slices), dim3(256), 0, st, a.g, x, a.x_ld,
                         a.A, a.r, a.K, part);
      constexpr int NB = RB <= 2 ? 2 : 1;
      hipLaunchKernelGGL((lora_few_wide_kernel<RB, NB>), dim3(tiles, (unsigned)div_up(a.N, 128 * NB)), dim3(256), 0, st,
                         a.g, part, slices, part == u ? nullptr : u, a.B, a.scale, a.r, a.N, base, y, a.y_ld);
    });
    return launched();
  }
  const int slice = narrow_slice(s, a.K), slices = div_up(a.K, slice);
  float* part = slices == 1 && u ? u : static_cast<float*>(ws);
  narrow<false>(a.g, s, x, a.x_ld, a.A, a.K, slice, part, st);
  wide<false>(a.g, s, part, slices, part == u ? nullptr : u, a.B, a.N, a.scale, base, y, a.y_ld, st);
  return launched();
}

moe_status_t launch_lora_bwd(const LoraArgs& a, const uint16_t* dy, const uint16_t* x, const float* u,
                             const uint16_t* dx_base, uint16_t* dx, float* dA, float* dB, int accumulate, void* ws,
                             hipStream_t st) {
  const LoraShape s = {a.g.M_cap, a.g.L, a.r, a.K, a.N};
  if (a.g.M_cap == 0 || a.g.T == 0) {          // no rows: the gradients of the adapters are 0
    if (!accumulate)
      for (int i = 0; i < 2; ++i) {
        float* p = i ? dB : dA;
        const long long n = (long long)a.g.L * a.r * (i ? a.N : a.K);
        if (p)
          hipLaunchKernelGGL(lora_zero_kernel, dim3((unsigned)(n < (1 << 20) ? div_up(n, 256) : 4096)), dim3(256), 0, st,
                             p, n);
      }
    return report(a.g, st);
  }
  const BwdLayout l = bwd_layout(s);
  char* base = static_cast<char*>(ws);
  float* w = reinterpret_cast<float*>(base + l.w);
  const int piece = sum_piece(s);
  const LoraSum sa = {w, x, a.x_ld, a.K, dA, reinterpret_cast<float*>(base + l.sumA)};
  const LoraSum sb = {u, dy, a.y_ld, a.N, dB, reinterpret_cast<float*>(base + l.sumB)};
  const auto sums = [&](bool wa, bool wb) {
    const int na = wa ? sum_blocks(s.r, a.K) : 0, nb = wb ? sum_blocks(s.r, a.N) : 0;
    if (na + nb == 0) return;
    const dim3 grid((unsigned)((s.M_cap / piece + s.L) * (na + nb)));
    for_rank_blocks(s.r, [&](auto n) {
      constexpr int RB = decltype(n)::value;
      hipLaunchKernelGGL((lora_sum_kernel<RB, RB <= 4 ? 8 : 4>), grid, dim3(256), 0, st, a.g, sa, sb, na, na + nb, a.scale, s.r,
                         piece, accumulate);
    });
  };
  if (dx && fused_back(s)) {
    few<true>(a.g, s, dy, a.y_ld, a.B, a.A, a.N, a.K, a.scale, dx_base, dx, a.x_ld, dA ? w : nullptr, st);
    sums(dA != nullptr, dB != nullptr);
  } else if (dx || dA) {
    int slice = narrow_slice(s, a.N);
    if (!dx) slice = div_up(a.N, 128) * 128;    // nothing adds slices up: one
    const int slices = div_up(a.N, slice);
    float* part = slices == 1 ? w : reinterpret_cast<float*>(base + l.narrow);
    narrow<true>(a.g, s, dy, a.y_ld, a.B, a.N, slice, part, st);
    if (dx) wide<true>(a.g, s, part, slices, part == w ? nullptr : w, a.A, a.K, a.scale, dx_base, dx, a.x_ld, st);
    sums(dA != nullptr, dB != nullptr);
  } else {
    if (report(a.g, st) != MOE_OK) return MOE_ERR_LAUNCH;
    sums(false, dB != nullptr);
  }
  if ((dA || dB) && many_groups(s) > 0) {
    const int ja = dA ? div_up((long long)s.r * a.K, 1024) : 0, jb = dB ? div_up((long long)s.r * a.N, 1024) : 0;
    hipLaunchKernelGGL(lora_join_kernel, dim3((unsigned)(ja + jb), (unsigned)many_groups(s)), dim3(256), 0, st, a.g, sa, sb,
                       ja, s.r, piece, accumulate);
  }
  return launched();
}

}  // namespace moe
