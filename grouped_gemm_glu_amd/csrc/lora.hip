// Launchers of the adapter kernels.
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
int narrow_slice(const LoraShape& s, int K) { return slice_of(K, tile_guess(s.M_cap, s.L, 64 * narrow_blocks(s)), 640); }
int wide_slice(const LoraShape& s, int N) {
  return slice_of(N, tile_guess(s.M_cap, s.L, 64), s.r > 64 ? 512 : 832);
}
size_t partial_bytes(const LoraShape& s, int K) {
  return aligned((size_t)div_up(K, narrow_slice(s, K)) * (size_t)s.M_cap * (size_t)s.r * 4);
}
int sum_blocks(int r, int C) { return div_up(C, r <= 64 ? 512 : 256); }
// Rows per workgroup of the sums, a multiple of 64, for about 512 workgroups.
int sum_piece(const LoraShape& s) {
  const long long p = (long long)s.M_cap * (sum_blocks(s.r, s.K) + sum_blocks(s.r, s.N)) / 512;
  return p <= 128 ? 128 : p >= kLoraPiece ? kLoraPiece : div_up(p, 64) * 64;
}
// Pieces of groups that have more than one: ceil(m / p) <= 2 m / p for m > p.
size_t sum_slots(const LoraShape& s) { return 2 * (size_t)s.M_cap / (size_t)sum_piece(s); }
// Whether a call of the forward goes by tiles of 16 rows.
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

moe_status_t report(const LoraGroups& g, hipStream_t st) {
  if (g.offsets_out || g.status_out) hipLaunchKernelGGL(lora_report_kernel, dim3(1), dim3(64), 0, st, g);
  return launched();
}
}  // namespace

size_t lora_fwd_workspace(const LoraShape& s) {
  return few_rows(s) ? aligned((size_t)div_up(s.K, 512) * (size_t)s.M_cap * (size_t)s.r * 4) : partial_bytes(s, s.K);
}
size_t lora_bwd_workspace(const LoraShape& s) { return bwd_layout(s).end; }

moe_status_t launch_lora_fwd(const LoraArgs& a, const uint16_t* x, const uint16_t* base, uint16_t* y, float* u,
                             void* ws, hipStream_t st) {
  const LoraShape s = {a.g.M_cap, a.g.L, a.r, a.K, a.N};
  if (a.g.M_cap == 0 || a.g.T == 0) return report(a.g, st);
  if (few_rows(s)) {
    const int slices = div_up(a.K, 512);
    const unsigned tiles = tile_bound(s.M_cap, s.L, 16);
    float* part = slices == 1 && u ? u : static_cast<float*>(ws);
    for_rank_blocks(s.r, [&](auto n) {
      constexpr int RB = decltype(n)::value;
      hipLaunchKernelGGL((lora_few_narrow_kernel<RB>), dim3(tiles, (unsigned)slices), dim3(256), 0, st, a.g, x, a.x_ld,
                         a.A, a.r, a.K, part);
      hipLaunchKernelGGL((lora_few_wide_kernel<RB, RB <= 2 ? 2 : 1>), dim3(tiles, (unsigned)div_up(a.N, RB <= 2 ? 256 : 128)), dim3(256), 0, st, a.g,
                         part, slices, part == u ? nullptr : u, a.B, a.scale, a.r, a.N, base, y, a.y_ld);
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
  if (dx || dA) {
    int slice = narrow_slice(s, a.N);
    if (!dx) slice = div_up(a.N, 128) * 128;    // nothing adds slices up: one
    const int slices = div_up(a.N, slice);
    float* part = slices == 1 ? w : reinterpret_cast<float*>(base + l.narrow);
    narrow<true>(a.g, s, dy, a.y_ld, a.B, a.N, slice, part, st);
    if (dx) wide<true>(a.g, s, part, slices, part == w ? nullptr : w, a.A, a.K, a.scale, dx_base, dx, a.x_ld, st);
  }
  if (!dx && !dA && report(a.g, st) != MOE_OK) return MOE_ERR_LAUNCH;
  if (dA || dB) {
    const int piece = sum_piece(s);
    const LoraSum sa = {w, x, a.x_ld, a.K, dA, reinterpret_cast<float*>(base + l.sumA), 0};
    const LoraSum sb = {u, dy, a.y_ld, a.N, dB, reinterpret_cast<float*>(base + l.sumB), 1};
    const int na = dA ? sum_blocks(s.r, a.K) : 0, nb = dB ? sum_blocks(s.r, a.N) : 0;
    const dim3 grid((unsigned)(s.M_cap / piece + s.L), (unsigned)(na + nb));
    for_rank_blocks(s.r, [&](auto n) {
      constexpr int RB = decltype(n)::value;
      hipLaunchKernelGGL((lora_sum_kernel<RB, RB <= 4 ? 8 : 4>), grid, dim3(256), 0, st, a.g, sa, sb, na, a.scale, s.r,
                         piece, accumulate);
    });
    if (s.M_cap > piece) {
      const int ja = dA ? div_up((long long)s.r * a.K, 1024) : 0, jb = dB ? div_up((long long)s.r * a.N, 1024) : 0;
      const int groups = s.M_cap / (piece + 1) < s.L ? s.M_cap / (piece + 1) : s.L;   // of more rows than a piece
      if (groups > 0)
        hipLaunchKernelGGL(lora_join_kernel, dim3((unsigned)(ja + jb), (unsigned)groups), dim3(256), 0, st, a.g, sa, sb,
                           ja, s.r, piece, accumulate);
    }
  }
  return launched();
}

}  // namespace moe
