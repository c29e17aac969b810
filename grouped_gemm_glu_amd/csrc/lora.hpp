// Low-rank adapters beside a shared projection: for the rows i of group e
//   u_i = A_e x_i            (the narrow product, rank r)
//   y_i = base_i + s_e B_e u_i
// and their gradients.  With w_i = B_e^T dy_i these are the same two products
// again (dx_i = base_i + s_e A_e^T w_i) and two sums over a group's rows
// (dA_e = s_e sum w_i x_i^T, dB_e = s_e sum dy_i u_i^T).  r is 8 to 128 where the
// rows are thousands long, so all of them are bound by memory: each row of x,
// y, dy and dx is read or written once, by MFMA fragments that lanes load and
// store directly.
//
// v_mfma_f32_16x16x32_bf16: lane l holds row (or column) l % 16 and the eight k
// from 8 (l / 16) on of each operand, and of the product column l % 16 and
// rows 4 (l / 16) .. + 3.
#pragma once

#include "device_common.hpp"
#include "operator_args.hpp"

namespace moe {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- tiles of the groups
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t lora_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
// Inclusive prefix over the wave's lanes of values up to cap < 2^31, each sum
// cut at cap: shifts within the rows of 16 lanes, then lane 15 of rows 0 and 2
// to rows 1 and 3, lane 31 to rows 2 and 3.
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v, uint32_t cap) {
  v = min(v + lora_dpp<0x111>(v), cap);
  v = min(v + lora_dpp<0x112>(v), cap);
  v = min(v + lora_dpp<0x114>(v), cap);
  v = min(v + lora_dpp<0x118>(v), cap);
  v = min(v + lora_dpp<0x142, 0xA>(v), cap);
  v = min(v + lora_dpp<0x143, 0xC>(v), cap);
  return v;
}
__device__ __forceinline__ int of_lane(uint32_t v, int lane) { return __builtin_amdgcn_readlane((int)v, lane); }

// A piece of a group: grouped rows [row, row + rows).
struct LoraTile {
  int e;        // group; -1: there is no such piece
  int row, rows;
  int index;    // piece of its group
  int pieces;   // of its group
  int slot;     // pieces before it of groups that have more than one
};

// Piece number `tile` when every group is cut into pieces of bm rows, a group
// without rows into `least` of none.  Each wave finds it for itself, without LDS
// or barriers: the groups' counts are cut so that they fit M_cap (a negative one
// is none), lanes hold PER of them each.
template <int PER>
__device__ __forceinline__ LoraTile find_piece(const LoraGroups& g, int bm, int least, uint32_t tile) {
  const int lane = threadIdx.x & 63;
  const uint32_t cap = (uint32_t)g.M_cap;
  uint32_t c[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    const int v = e < g.L ? g.counts[e] : 0;
    c[i] = min((uint32_t)(v < 0 ? 0 : v), cap);
    sum = min(sum + c[i], cap);
  }
  const uint32_t incl = wave_prefix(sum, cap);
  // the lanes before this one: exact while they fit, else cap
  uint32_t run = lora_dpp<0x138>(incl);   // from the lane before (wave_shr:1)
  if (lane == 0) run = 0;
  const uint32_t first = run;
  uint32_t pieces = 0, many = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = min(c[i], cap - run);
    run += c[i];
    const uint32_t n = lane * PER + i < g.L ? max((c[i] + bm - 1) / bm, (uint32_t)least) : 0;
    pieces += n;
    many += n > 1 ? n : 0;
  }
  constexpr uint32_t kNoCap = 0x7FFFFFFF;
  const uint32_t pi = wave_prefix(pieces, kNoCap), mi = wave_prefix(many, kNoCap);
  const unsigned long long past = __ballot(pi > tile);
  LoraTile t;
  t.e = -1;
  if (past == 0) return t;
  const int at = __builtin_ctzll(past);
  // the lane that holds the piece walks its groups
  uint32_t before = pi - pieces, slot = mi - many, row = first;
  int e = 0, rows = 0, index = 0, n_of = 0, start = 0, base = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t n = lane * PER + i < g.L ? max((c[i] + bm - 1) / bm, (uint32_t)least) : 0;
    if (!found && tile - before < n) {
      found = true;
      index = (int)(tile - before);
      e = lane * PER + i;
      n_of = (int)n;
      start = (int)row + index * bm;
      rows = min(bm, (int)c[i] - index * bm);
      base = (int)slot + index;
    }
    before += n;
    slot += n > 1 ? n : 0;
    row += c[i];
  }
  t.e = of_lane(e, at);
  t.row = of_lane(start, at);
  t.rows = of_lane(rows, at);
  t.index = of_lane(index, at);
  t.pieces = of_lane(n_of, at);
  t.slot = of_lane(base, at);
  return t;
}
__device__ __forceinline__ LoraTile lora_tile(const LoraGroups& g, int bm, int least, uint32_t tile) {
  return g.L <= 64 ? find_piece<1>(g, bm, least, tile) : find_piece<kMaxExperts / 64>(g, bm, least, tile);
}

// offsets_out and status_out of moe_groups_t, by one wave.
__device__ inline void lora_report(const LoraGroups& g) {
  if (!g.offsets_out && !g.status_out) return;
  const int lane = threadIdx.x & 63;
  constexpr int PER = kMaxExperts / 64;
  long long sum = 0;
  int bad = 0;
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    const int v = e < g.L ? g.counts[e] : 0;
    bad |= v < 0;
    sum += v < 0 ? 0 : v;
  }
  long long incl = sum;
  for (int d = 1; d < 64; d <<= 1) {
    const long long o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  long long run = incl - sum;
  if (g.offsets_out) {
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      if (e < g.L) {
        const int v = g.counts[e];
        g.offsets_out[e] = (int)(run < g.M_cap ? run : g.M_cap);
        run += v < 0 ? 0 : v;
        if (e == g.L - 1) g.offsets_out[g.L] = (int)(run < g.M_cap ? run : g.M_cap);
      }
    }
  }
  const int any_bad = __any(bad);
  if (g.status_out && lane == 63) {
    const int st = (any_bad ? 1 : 0) | (incl > g.M_cap ? 2 : 0);
    if (st) atomicOr(g.status_out, st);
  }
}

__global__ __launch_bounds__(64) void lora_report_kernel(LoraGroups g) { lora_report(g); }

// The row of x and y that grouped row g is; -1: none (no such row).
__device__ __forceinline__ int lora_row(const LoraGroups& g, int grow, bool inside) {
  if (!inside) return -1;
  const int r = g.src ? g.src[grow] : grow;
  return r >= 0 && r < g.T ? r : -1;
}

__device__ __forceinline__ bf16x8 load8(const uint16_t* p) {
  return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(p));
}
__device__ __forceinline__ bf16x8 zero8() {
  const u32x4 z = {0, 0, 0, 0};
  return __builtin_bit_cast(bf16x8, z);
}

// ---------------------------------------------------------------- u = x A^T
// A tile of 16 MB rows and a slice of K per workgroup; its four waves take runs
// of 128 columns in turn and their sums meet in LDS.  The slices' sums go to
// out + slice * M_cap * r (one slice: the result itself); the next kernel adds
// them in that order.  Rows that src does not name get 0.
template <int RB, int MB>
__global__ __launch_bounds__(256) void lora_narrow_kernel(LoraGroups g, const uint16_t* __restrict__ x, long long x_ld,
                                                          const uint16_t* __restrict__ A, int r, int K, int slice,
                                                          float* __restrict__ out, bool report) {
  constexpr int BM = 16 * MB, RP = 16 * RB, LD = RP + 4;
  __shared__ float red[4 * BM * LD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row16 = lane & 15, q = lane >> 4;
  if (report && blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) lora_report(g);
  const LoraTile t = lora_tile(g, BM, 0, blockIdx.x);
  if (t.e < 0) return;
  const uint16_t* xr[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int at = 16 * m + row16;
    const int row = lora_row(g, t.row + at, at < t.rows);
    xr[m] = x + (long long)max(row, 0) * x_ld;   // a row that is none: any, its sums are dropped
  }
  const uint16_t* ar[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) ar[b] = A + ((long long)t.e * r + min(16 * b + row16, r - 1)) * K;
  const int k_end = min(K, (int)(blockIdx.y + 1) * slice);
  f32x4 acc[MB][RB] = {};
  for (int k0 = blockIdx.y * slice + 128 * wave; k0 < k_end; k0 += 512) {
    if (k0 + 128 <= k_end) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 32 * j + 8 * q;
        bf16x8 xv[MB], av[RB];
#pragma unroll
        for (int m = 0; m < MB; ++m) xv[m] = load8(xr[m] + k);
#pragma unroll
        for (int b = 0; b < RB; ++b) av[b] = load8(ar[b] + k);
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int b = 0; b < RB; ++b)
            acc[m][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[b], xv[m], acc[m][b], 0, 0, 0);
      }
    } else {
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 32 * j + 8 * q;
        const bool in = k < k_end;               // slices and K are multiples of 8
        bf16x8 xv[MB], av[RB];
#pragma unroll
        for (int m = 0; m < MB; ++m) xv[m] = in ? load8(xr[m] + k) : zero8();
#pragma unroll
        for (int b = 0; b < RB; ++b) av[b] = in ? load8(ar[b] + k) : zero8();
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int b = 0; b < RB; ++b)
            acc[m][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[b], xv[m], acc[m][b], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int b = 0; b < RB; ++b)
      *reinterpret_cast<f32x4*>(&red[(wave * BM + 16 * m + row16) * LD + 16 * b + 4 * q]) = acc[m][b];
  __syncthreads();
  float* o = out + (long long)blockIdx.y * g.M_cap * r;
  const int quads = r / 4;
  for (int i = threadIdx.x; i < t.rows * quads; i += 256) {
    const int row = i / quads, c = 4 * (i - row * quads);
    f32x4 s = *reinterpret_cast<const f32x4*>(&red[row * LD + c]);
#pragma unroll
    for (int w = 1; w < 4; ++w) s += *reinterpret_cast<const f32x4*>(&red[(w * BM + row) * LD + c]);
    if (lora_row(g, t.row + row, true) < 0) s = f32x4{0, 0, 0, 0};
    *reinterpret_cast<f32x4*>(o + (long long)(t.row + row) * r + c) = s;
  }
}

// ---------------------------------------------------------------- y = base + s u B^T
// fp32 as a sum of bf16 values: the upper half of its bits (no rounding, so that
// nothing overflows), then what is left.  Two parts hold a value to 2^-17, far
// below the bf16 rounding of y; an infinity is its first part alone.
__device__ __forceinline__ uint32_t upper_half(float v) { return __float_as_uint(v) >> 16; }
__device__ __forceinline__ float rest_of(float v) {
  const float hi = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
  return v == hi ? 0.0f : v - hi;
}

// A tile of 16 MB rows and a slice of N per workgroup.  The rows' u (the slices'
// sums added in order, times s) is staged in LDS as its two bf16 parts, [upper r
// | rest r | zeros], which is one reduction of KS MFMA steps against the weight
// row taken twice.  A wave takes 32 columns at a time: the rows of two MFMAs are
// chosen so that a lane's eight products are eight consecutive columns.
template <int KS, int MB>
__global__ __launch_bounds__(256) void lora_wide_kernel(LoraGroups g, const float* __restrict__ u_in, int slices,
                                                        float* __restrict__ u_out, const uint16_t* __restrict__ B,
                                                        const float* __restrict__ scale, int r, int N, int slice,
                                                        const uint16_t* base, uint16_t* y, long long y_ld) {
  constexpr int BM = 16 * MB, LD = 32 * KS + 8;
  __shared__ __attribute__((aligned(16))) uint16_t us[BM * LD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row16 = lane & 15, q = lane >> 4;
  const LoraTile t = lora_tile(g, BM, 0, blockIdx.x);
  if (t.e < 0) return;
  const float s = scale ? scale[t.e] : 1.0f;
  const int quads = r / 4;
  for (int i = threadIdx.x; i < BM * 8 * KS; i += 256) {   // 4 r of a row, zeros past the two parts
    const int row = i / (8 * KS), c = i - row * (8 * KS);
    if (c < quads) {
      f32x4 v = {0, 0, 0, 0};
      if (row < t.rows) {
        const float* p = u_in + (long long)(t.row + row) * r + 4 * c;
        v = *reinterpret_cast<const f32x4*>(p);
        for (int k = 1; k < slices; ++k) v += *reinterpret_cast<const f32x4*>(p + (long long)k * g.M_cap * r);
        if (u_out && blockIdx.y == 0) *reinterpret_cast<f32x4*>(u_out + (long long)(t.row + row) * r + 4 * c) = v;
      }
      v *= s;
      uint2 hi, lo;
      hi.x = upper_half(v[0]) | upper_half(v[1]) << 16;
      hi.y = upper_half(v[2]) | upper_half(v[3]) << 16;
      lo.x = pack_bf16x2(rest_of(v[0]), rest_of(v[1]));
      lo.y = pack_bf16x2(rest_of(v[2]), rest_of(v[3]));
      *reinterpret_cast<uint2*>(&us[row * LD + 4 * c]) = hi;
      *reinterpret_cast<uint2*>(&us[row * LD + r + 4 * c]) = lo;
    } else if (c >= 2 * quads) {
      *reinterpret_cast<uint2*>(&us[row * LD + 4 * c]) = make_uint2(0, 0);
    }
  }
  __syncthreads();
  bf16x8 uv[MB][KS];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int k = 0; k < KS; ++k) uv[m][k] = load8(&us[(16 * m + row16) * LD + 32 * k + 8 * q]);
  int at[KS];             // this lane's place in a weight row at each step; -1: past both parts
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const int c = 8 * (4 * k + q);
    at[k] = c < r ? c : c < 2 * r ? c - r : -1;
  }
  long long yo[MB];
  bool there[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int i = 16 * m + row16;
    const int row = lora_row(g, t.row + i, i < t.rows);
    there[m] = row >= 0;
    yo[m] = (long long)max(row, 0) * y_ld;
  }
  const uint16_t* Be = B + (long long)t.e * N * r;
  const int n_end = min(N, (int)(blockIdx.y + 1) * slice);
  const int nw = 8 * (row16 >> 2) + (row16 & 3);   // weight row of the first MFMA; the second's: + 4
  for (int n0 = blockIdx.y * slice + 32 * wave; n0 < n_end; n0 += 128) {
    f32x4 acc[MB][2] = {};
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = min(n0 + nw + 4 * j, N - 1);
        const bf16x8 bv = at[k] >= 0 ? load8(Be + (long long)n * r + at[k]) : zero8();
#pragma unroll
        for (int m = 0; m < MB; ++m)
          acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, uv[m][k], acc[m][j], 0, 0, 0);
      }
    const int n = n0 + 8 * q;
    if (n < n_end)
#pragma unroll
      for (int m = 0; m < MB; ++m)
        if (there[m]) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = acc[m][i >> 2][i & 3];
          if (base) {
            const u32x4 b = *reinterpret_cast<const u32x4*>(base + yo[m] + n);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[2 * i] += __uint_as_float(b[i] << 16);
              v[2 * i + 1] += __uint_as_float(b[i] & 0xFFFF0000u);
            }
          }
          u32x4 o;
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
          *reinterpret_cast<u32x4*>(y + yo[m] + n) = o;
        }
  }
}

// ---------------------------------------------------------------- weights turned round
// dst[c][r] = src[r][c] (rows x cols), for the groups that have rows: the
// backward's products read the adapters in the forward's layout.  A tile of 64 x
// 64 through LDS.
__global__ __launch_bounds__(256) void lora_turn_kernel(LoraGroups g, const uint16_t* __restrict__ src, int rows,
                                                        int cols, uint16_t* __restrict__ dst) {
  __shared__ uint16_t tile[64][66];
  const int e = blockIdx.z;
  if (g.counts[e] <= 0) return;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const uint16_t* s = src + (long long)e * rows * cols;
  uint16_t* d = dst + (long long)e * rows * cols;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int r = i >> 6, c = i & 63;
    if (r0 + r < rows && c0 + c < cols) tile[r][c] = s[(long long)(r0 + r) * cols + c0 + c];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int c = i >> 6, r = i & 63;
    if (r0 + r < rows && c0 + c < cols) d[(long long)(c0 + c) * rows + r0 + r] = tile[r][c];
  }
}

// ---------------------------------------------------------------- dA, dB
// The sums over a group's rows of (s u_i) v_i^T, u fp32 [M_cap][r], v bf16 rows of
// C columns: dA from w and x, dB from u and dy.  A piece of at most `piece` rows
// of a group and a block of 16 CW columns per workgroup, whose four waves take 32
// rows in turn; their sums meet in LDS.  The MFMA wants eight rows of one column
// per lane where memory has columns side by side: a lane loads CW columns of its
// eight rows and takes them apart with byte permutations, one MFMA for each.  u
// goes in as three bf16 parts, 24 bits of it, so that the sums are those of
// fp32 products.
struct LoraSum {
  const float* u;
  const uint16_t* v;
  long long v_ld;
  int C;
  float* out;        // [L][r][C], or [L][C][r] with turned
  float* part;       // [slots][r][C] likewise, of groups of more than one piece
  int turned;
};

__device__ __forceinline__ uint32_t pick16(uint32_t lo, uint32_t hi, bool upper) {
  return __builtin_amdgcn_perm(hi, lo, upper ? 0x07060302u : 0x05040100u);
}

template <int RB, int CW>
__global__ __launch_bounds__(256) void lora_sum_kernel(LoraGroups g, LoraSum a, LoraSum b, int a_blocks,
                                                       const float* __restrict__ scale, int r, int piece,
                                                       int accumulate) {
  __shared__ float red[2 * RB * CW * 4 * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row16 = lane & 15, q = lane >> 4;
  const LoraTile t = lora_tile(g, piece, accumulate ? 0 : 1, blockIdx.x);
  if (t.e < 0) return;
  const bool first = (int)blockIdx.y < a_blocks;
  const LoraSum& p = first ? a : b;
  const int c0 = (first ? blockIdx.y : blockIdx.y - a_blocks) * 16 * CW;
  const int c = c0 + CW * row16;
  const bool col_in = c < p.C;                  // C is a multiple of 8
  const float s = scale ? scale[t.e] : 1.0f;
  f32x4 acc[RB][CW] = {};
  for (int i0 = 32 * wave; i0 < t.rows; i0 += 128) {
    uint32_t raw[8][CW / 2];
    int grow[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = i0 + 8 * q + i;
      grow[i] = t.row + at;
      const int row = lora_row(g, grow[i], at < t.rows);
      if (row < 0) grow[i] = -1;
#pragma unroll
      for (int w = 0; w < CW / 2; ++w) raw[i][w] = 0;
      if (row >= 0 && col_in) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.v + (long long)row * p.v_ld + c);
        if constexpr (CW == 8) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(src);
          raw[i][0] = v[0]; raw[i][1] = v[1]; raw[i][2] = v[2]; raw[i][3] = v[3];
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(src);
          raw[i][0] = v.x; raw[i][1] = v.y;
        }
      }
    }
    bf16x8 col[CW];
#pragma unroll
    for (int j = 0; j < CW; ++j) {
      u32x4 f;
#pragma unroll
      for (int d = 0; d < 4; ++d) f[d] = pick16(raw[2 * d][j / 2], raw[2 * d + 1][j / 2], j & 1);
      col[j] = __builtin_bit_cast(bf16x8, f);
    }
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      const int ri = 16 * k + row16;
      u32x4 p0, p1, p2;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        float v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int gr = grow[2 * d + h];
          v[h] = gr >= 0 && ri < r ? s * p.u[(long long)gr * r + ri] : 0.0f;
        }
        const float r0 = rest_of(v[0]), r1 = rest_of(v[1]);
        p0[d] = upper_half(v[0]) | upper_half(v[1]) << 16;
        p1[d] = upper_half(r0) | upper_half(r1) << 16;
        p2[d] = pack_bf16x2(rest_of(r0), rest_of(r1));
      }
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        acc[k][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p2), col[j], acc[k][j], 0, 0, 0);
        acc[k][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p1), col[j], acc[k][j], 0, 0, 0);
        acc[k][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p0), col[j], acc[k][j], 0, 0, 0);
      }
    }
  }
  // waves 2 and 3 onto 0 and 1, then 1 onto 0
  f32x4* box = reinterpret_cast<f32x4*>(red);
#pragma unroll
  for (int step = 2; step >= 1; step >>= 1) {
    if (wave >= step && wave < 2 * step)
#pragma unroll
      for (int k = 0; k < RB; ++k)
#pragma unroll
        for (int j = 0; j < CW; ++j) box[(((wave - step) * RB + k) * CW + j) * 64 + lane] = acc[k][j];
    __syncthreads();
    if (wave < step)
#pragma unroll
      for (int k = 0; k < RB; ++k)
#pragma unroll
        for (int j = 0; j < CW; ++j) acc[k][j] += box[((wave * RB + k) * CW + j) * 64 + lane];
    __syncthreads();
  }
  if (wave != 0 || !col_in) return;
  const bool whole = t.pieces == 1;
  float* o = (whole ? p.out + (long long)t.e * r * p.C : p.part + (long long)t.slot * r * p.C);
  const bool add = whole && accumulate;
#pragma unroll
  for (int k = 0; k < RB; ++k) {
    const int ri = 16 * k + 4 * q;              // r is a multiple of 8: all four or none
    if (ri >= r) continue;
    if (p.turned) {
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        f32x4* d = reinterpret_cast<f32x4*>(o + (long long)(c + j) * r + ri);
        *d = add ? *d + acc[k][j] : acc[k][j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < CW; j += 4) {
          f32x4* d = reinterpret_cast<f32x4*>(o + (long long)(ri + i) * p.C + c + j);
          const f32x4 v = {acc[k][j][i], acc[k][j + 1][i], acc[k][j + 2][i], acc[k][j + 3][i]};
          *d = add ? *d + v : v;
        }
    }
  }
}

// The pieces of the groups that have more than one, added in their order.
__global__ __launch_bounds__(256) void lora_join_kernel(LoraGroups g, LoraSum a, LoraSum b, int a_blocks, int r,
                                                        int piece, int accumulate) {
  // the first piece of group e, found by walking to it
  const int e = blockIdx.x;
  const int lane = threadIdx.x & 63;
  long long run = 0;
  int slot = 0, mine = 0;
  for (int f0 = 0; f0 <= e; f0 += 64) {
    // 64 counts at a time, every lane walks them
    const int f = f0 + lane;
    const int v = f < g.L ? g.counts[f] : 0;
    for (int i = 0; i < 64 && f0 + i <= e; ++i) {
      const int c = __builtin_amdgcn_readlane(v, i);
      const long long room = g.M_cap - run;
      const int m = c <= 0 || room <= 0 ? 0 : (int)(c < room ? c : room);
      run += c < 0 ? 0 : c;
      const int n = (m + piece - 1) / piece;
      if (f0 + i == e) mine = n;
      else slot += n > 1 ? n : 0;
    }
  }
  if (mine <= 1) return;
  const bool first = (int)blockIdx.y < a_blocks;
  const LoraSum& p = first ? a : b;
  const long long size = (long long)r * p.C;
  const long long i = 4 * ((long long)(first ? blockIdx.y : blockIdx.y - a_blocks) * 256 + threadIdx.x);
  if (i >= size) return;
  const float* src = p.part + (long long)slot * size + i;
  f32x4 s = *reinterpret_cast<const f32x4*>(src);
  for (int k = 1; k < mine; ++k) s += *reinterpret_cast<const f32x4*>(src + (long long)k * size);
  f32x4* d = reinterpret_cast<f32x4*>(p.out + (long long)e * size + i);
  *d = accumulate ? *d + s : s;
}

// Zeros for the gradients of a call without rows.
__global__ __launch_bounds__(256) void lora_zero_kernel(float* p, long long n) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) p[i] = 0.0f;
}

}  // namespace moe
