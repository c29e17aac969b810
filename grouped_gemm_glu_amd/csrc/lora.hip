// Launchers of the adapter kernels.
#include "internal.hpp"
#include "lora.hpp"

namespace moe {

namespace {
moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }
int div_up(long long a, long long b) { return (int)((a + b - 1) / b); }
size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

// 16-row blocks per tile
int tile_blocks(int M_cap, int L) { return M_cap <= 16LL * L ? 1 : 2; }
// An upper bound of the tiles: each group adds at most one partial tile.
unsigned tile_bound(int M_cap, int L, int bm) { return (unsigned)(M_cap / bm + (L < M_cap ? L : M_cap)); }
// Columns per workgroup, a multiple of step, for about `target` workgroups.
int slice_of(int cols, int tiles, int step, int target) {
  int n = target / (tiles > 0 ? tiles : 1);
  n = n < 1 ? 1 : n;
  const int s = div_up(div_up(cols, n), step) * step;
  return s;
}
int narrow_slice(const LoraShape& s, int K) {
  return slice_of(K, s.M_cap / (16 * tile_blocks(s.M_cap, s.L)), 512, 1024);
}
int wide_slice(const LoraShape& s, int N) {
  return slice_of(N, s.M_cap / (16 * tile_blocks(s.M_cap, s.L)), 128, 2048);
}
size_t partial_bytes(const LoraShape& s, int K) {
  return aligned((size_t)div_up(K, narrow_slice(s, K)) * (size_t)s.M_cap * (size_t)s.r * 4);
}
// columns per lane of the sums
int sum_cols(int r) { return r <= 64 ? 8 : 4; }
int sum_blocks(const LoraShape& s, int C) { return div_up(C, 16 * sum_cols(s.r)); }
// Rows per workgroup of the sums: a power of two, for about 1024 workgroups.
int sum_piece(const LoraShape& s) {
  const long long blocks = sum_blocks(s, s.K) + sum_blocks(s, s.N);
  int p = 128;
  while (p < (1 << 20) && p < s.M_cap * blocks / 1024) p *= 2;
  return p;
}
// Pieces of groups that have more than one: ceil(m / p) <= 2 m / p for m > p.
size_t sum_slots(const LoraShape& s) { return 2 * (size_t)s.M_cap / (size_t)sum_piece(s); }

template <typename F>
void for_rank_blocks(int r, F&& f) {
  if (r <= 16) f(std::integral_constant<int, 1>{});
  else if (r <= 32) f(std::integral_constant<int, 2>{});
  else if (r <= 64) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 8>{});
}

struct BwdLayout {
  size_t At, Bt, w, narrow, sumA, sumB, end;
};
BwdLayout bwd_layout(const LoraShape& s) {
  BwdLayout l;
  const size_t a = (size_t)s.L * s.r * s.K, b = (size_t)s.L * s.r * s.N;
  l.At = 0;
  l.Bt = l.At + aligned(2 * a);
  l.w = l.Bt + aligned(2 * b);
  l.narrow = l.w + aligned((size_t)s.M_cap * s.r * 4);
  l.sumA = l.narrow + partial_bytes(s, s.N);
  l.sumB = l.sumA + aligned(sum_slots(s) * (size_t)s.r * s.K * 4);
  l.end = l.sumB + aligned(sum_slots(s) * (size_t)s.r * s.N * 4);
  return l;
}

void narrow(const LoraGroups& g, const LoraShape& s, const uint16_t* x, long long x_ld, const uint16_t* A, int K,
            int slice, float* out, bool report, hipStream_t st) {
  const int mb = tile_blocks(s.M_cap, s.L);
  const dim3 grid(tile_bound(s.M_cap, s.L, 16 * mb), (unsigned)div_up(K, slice));
  for_rank_blocks(s.r, [&](auto n) {
    constexpr int RB = decltype(n)::value;
    if (mb == 1)
      hipLaunchKernelGGL((lora_narrow_kernel<RB, 1>), grid, dim3(256), 0, st, g, x, x_ld, A, s.r, K, slice, out, report);
    else
      hipLaunchKernelGGL((lora_narrow_kernel<RB, 2>), grid, dim3(256), 0, st, g, x, x_ld, A, s.r, K, slice, out, report);
  });
}

void wide(const LoraGroups& g, const LoraShape& s, const float* u, int slices, float* u_out, const uint16_t* B, int N,
          const float* scale, const uint16_t* base, uint16_t* y, long long y_ld, hipStream_t st) {
  const int mb = tile_blocks(s.M_cap, s.L), slice = wide_slice(s, N);
  const dim3 grid(tile_bound(s.M_cap, s.L, 16 * mb), (unsigned)div_up(N, slice));
  for_rank_blocks(s.r, [&](auto n) {
    constexpr int KS = decltype(n)::value;
    if (mb == 1)
      hipLaunchKernelGGL((lora_wide_kernel<KS, 1>), grid, dim3(256), 0, st, g, u, slices, u_out, B, scale, s.r, N,
                         slice, base, y, y_ld);
    else
      hipLaunchKernelGGL((lora_wide_kernel<KS, 2>), grid, dim3(256), 0, st, g, u, slices, u_out, B, scale, s.r, N,
                         slice, base, y, y_ld);
  });
}

moe_status_t report(const LoraGroups& g, hipStream_t st) {
  if (g.offsets_out || g.status_out) hipLaunchKernelGGL(lora_report_kernel, dim3(1), dim3(64), 0, st, g);
  return launched();
}
}  // namespace

size_t lora_fwd_workspace(const LoraShape& s) { return partial_bytes(s, s.K); }
size_t lora_bwd_workspace(const LoraShape& s) { return bwd_layout(s).end; }

moe_status_t launch_lora_fwd(const LoraArgs& a, const uint16_t* x, const uint16_t* base, uint16_t* y, float* u,
                             void* ws, hipStream_t st) {
  const LoraShape s = {a.g.M_cap, a.g.L, a.r, a.K, a.N};
  if (a.g.M_cap == 0 || a.g.T == 0) return report(a.g, st);
  const int slice = narrow_slice(s, a.K), slices = div_up(a.K, slice);
  float* part = slices == 1 && u ? u : static_cast<float*>(ws);
  narrow(a.g, s, x, a.x_ld, a.A, a.K, slice, part, true, st);
  wide(a.g, s, part, slices, part == u ? nullptr : u, a.B, a.N, a.scale, base, y, a.y_ld, st);
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
  uint16_t* At = reinterpret_cast<uint16_t*>(base + l.At);
  uint16_t* Bt = reinterpret_cast<uint16_t*>(base + l.Bt);
  float* w = reinterpret_cast<float*>(base + l.w);
  if (dx || dA) {
    const auto turn = [&](const uint16_t* src, int rows, int cols, uint16_t* dst) {
      hipLaunchKernelGGL(lora_turn_kernel, dim3((unsigned)div_up(cols, 64), (unsigned)div_up(rows, 64), (unsigned)s.L),
                         dim3(256), 0, st, a.g, src, rows, cols, dst);
    };
    turn(a.B, a.N, a.r, Bt);
    if (dx) turn(a.A, a.r, a.K, At);
    int slice = narrow_slice(s, a.N);
    if (!dx) slice = div_up(a.N, 512) * 512;    // nothing adds slices up: one
    const int slices = div_up(a.N, slice);
    float* part = slices == 1 ? w : reinterpret_cast<float*>(base + l.narrow);
    narrow(a.g, s, dy, a.y_ld, Bt, a.N, slice, part, true, st);
    if (dx) wide(a.g, s, part, slices, part == w ? nullptr : w, At, a.K, a.scale, dx_base, dx, a.x_ld, st);
  }
  if (!dx && !dA && report(a.g, st) != MOE_OK) return MOE_ERR_LAUNCH;
  if (dA || dB) {
    const int piece = sum_piece(s);
    const LoraSum sa = {w, x, a.x_ld, a.K, dA, reinterpret_cast<float*>(base + l.sumA), 0};
    const LoraSum sb = {u, dy, a.y_ld, a.N, dB, reinterpret_cast<float*>(base + l.sumB), 1};
    const int na = dA ? sum_blocks(s, a.K) : 0, nb = dB ? sum_blocks(s, a.N) : 0;
    const dim3 grid((unsigned)(s.M_cap / piece + s.L), (unsigned)(na + nb));
    for_rank_blocks(s.r, [&](auto n) {
      constexpr int RB = decltype(n)::value;
      constexpr int CW = RB <= 4 ? 8 : 4;
      hipLaunchKernelGGL((lora_sum_kernel<RB, CW>), grid, dim3(256), 0, st, a.g, sa, sb, na, a.scale, s.r, piece,
                         accumulate);
    });
    if (s.M_cap > piece) {
      const int ja = dA ? div_up((long long)s.r * a.K, 1024) : 0, jb = dB ? div_up((long long)s.r * a.N, 1024) : 0;
      hipLaunchKernelGGL(lora_join_kernel, dim3((unsigned)s.L, (unsigned)(ja + jb)), dim3(256), 0, st, a.g, sa, sb, ja,
                         s.r, piece, accumulate);
    }
  }
  return launched();
}

}  // namespace moe
