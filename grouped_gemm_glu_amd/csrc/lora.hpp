// Low-rank adapters beside a shared projection: for the rows i of group e
//   u_i = A_e x_i            (the narrow product, rank r)
//   y_i = base_i + s_e B_e u_i
// and their gradients.  With w_i = B_e^T dy_i these are the same two products
// again (dx_i = base_i + s_e A_e^T w_i) and two sums over a group's rows
// (dA_e = s_e sum w_i x_i^T, dB_e = s_e sum dy_i u_i^T).  r is 8 to 128 where the
// rows are thousands long, so memory is the floor of all of them (what keeps each
// above it stands there): a row of x, y, dy and dx is read or written once a kernel.
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
  int pieces;   // of its group
  int slot;     // pieces before it of groups that have more than one
};

// Piece number `tile` when every group is cut into pieces of bm rows, a group
// without rows into `least` of none; with MANY the tile-th of the groups that have
// more than one piece (its first).  Each wave finds it for itself, without LDS or
// barriers: the groups' counts are cut so that they fit M_cap (a negative one is
// none), lanes hold PER of them each.  With PER 16 (more than 64 groups) the counts are
// loaded one after the other: a call of 64 rows in 64 groups 8.8 us, in 65 10.9, in 1024
// 13.2 (r 16, K 2880, N 5760).
template <int PER, bool MANY, bool EVEN>
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
    pieces += MANY ? n > 1 : n;
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
  int e = 0, rows = 0, n_of = 0, start = 0, base = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t n = lane * PER + i < g.L ? max((c[i] + bm - 1) / bm, (uint32_t)least) : 0;
    const uint32_t units = MANY ? n > 1 : n;
    if (!found && tile - before < units) {
      found = true;
      const int index = MANY ? 0 : (int)(tile - before);
      e = lane * PER + i;
      n_of = (int)n;
      const int len = EVEN && n > 0 ? ((int)((c[i] + n - 1) / n) + 31) / 32 * 32 : bm;
      start = (int)row + index * len;
      rows = min(len, (int)c[i] - index * len);
      base = (int)slot + index;
    }
    before += units;
    slot += n > 1 ? n : 0;
    row += c[i];
  }
  t.e = of_lane(e, at);
  t.row = of_lane(start, at);
  t.rows = of_lane(rows, at);
  t.pieces = of_lane(n_of, at);
  t.slot = of_lane(base, at);
  return t;
}
__device__ __forceinline__ LoraTile lora_tile(const LoraGroups& g, int bm, uint32_t tile) {
  return g.L <= 64 ? find_piece<1, false, false>(g, bm, 0, tile)
                   : find_piece<kMaxExperts / 64, false, false>(g, bm, 0, tile);
}
// pieces of at most bm rows (a multiple of 32), equal within a group but for 32 rows
__device__ __forceinline__ LoraTile lora_piece(const LoraGroups& g, int bm, int least, uint32_t tile) {
  return g.L <= 64 ? find_piece<1, false, true>(g, bm, least, tile)
                   : find_piece<kMaxExperts / 64, false, true>(g, bm, least, tile);
}
__device__ __forceinline__ LoraTile lora_many(const LoraGroups& g, int bm, uint32_t which) {
  return g.L <= 64 ? find_piece<1, true, false>(g, bm, 0, which)
                   : find_piece<kMaxExperts / 64, true, false>(g, bm, 0, which);
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

// fp32 as a sum of three bf16 values: the upper half of its bits, the same of what is
// left, and the rest, 8 bits each.  An infinity is its first part alone.
__device__ __forceinline__ uint32_t upper_half(float v) { return __float_as_uint(v) >> 16; }
__device__ __forceinline__ float rest_of(float v) {
  const float hi = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
  return v == hi ? 0.0f : v - hi;
}
// Two values as sums of two each: the nearest bf16 values, then what is left, half a step
// at most and rounded in its turn, 2^-17 of them (the upper half first would leave up to a
// whole step: 2^-16).  The first part is cut at bf16's largest value, so that nothing
// rounds up to an infinity; an infinity or a NaN is in the second.
struct TwoParts {
  uint32_t first, rest;
};
__device__ __forceinline__ TwoParts two_parts(float v0, float v1) {
  const float top = __uint_as_float(0x7F7F0000u);
  TwoParts p;
  p.first = pack_bf16x2(__builtin_amdgcn_fmed3f(v0, -top, top), __builtin_amdgcn_fmed3f(v1, -top, top));
  p.rest = pack_bf16x2(v0 - __uint_as_float(p.first << 16), v1 - __uint_as_float(p.first & 0xFFFF0000u));
  return p;
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A value that the compiler knows nothing of.  Where the lanes of a wave read one
// another's values from a piece of LDS that the wave has to itself, LDS works through
// its accesses in order, so nothing has to be waited for; but the compiler, which sees
// one lane, may swap a lane's write and read where it can prove them apart.  A read whose
// place follows from such a value it cannot tell from any write to the piece.  (Fences say
// the same, but hold loads from memory back too: 1 row, r 16, K 7168 8.1 us for 7.7.)
__device__ __forceinline__ int hidden(int v) {
  asm("" : "+v"(v));
  return v;
}

// Four consecutive elements of each of four rows of LDS, crosswise: in every 16
// lanes, lane l gives the address of row l / 4, elements 4 (l % 4) .. + 3, and
// gets element l of the four rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x8 read_crosswise(const uint16_t* rows0, const uint16_t* rows4) {
  typedef __attribute__((address_space(3))) s16x4* lds_t;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)rows0);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)rows4);
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// ---------------------------------------------------------------- u = x W^T
// A tile of 64 MB rows and a slice of K per workgroup, 128 columns of K at a
// time, the next step's x and the weights after it in flight.  A wave loads its 16 MB rows as
// runs of 256 bytes (16 lanes a row) and turns them into fragments through a piece
// of LDS of its own; the weights come through LDS for all waves (two stages), so
// that a row block reads them once.  W is [r][K], or with TURNED [K][r] (the
// backward's w = dy B), whose fragments are read crosswise.  The slices' sums go
// to out + slice * M_cap * r (one slice: the result itself); the next kernel adds
// them in that order.  Rows that src does not name get 0.
//
// Measured: 14746 rows, r 64, K 7168 62 us (51 where nothing else uses the memory, 4.1
// TB/s); 16384 rows in 32 groups, r 32 69 us, 3.4 TB/s, of which a fifth is what the kernel
// before it wrote on its way to memory; 8191 rows, r 16, K 2880 17 us, a third of it the
// start (counts, src, the first rows); 8192 rows, r 128, K 7168 68 us, 1.7 TB/s, where the
// LDS holds one workgroup to a compute unit.  Blocks of 256 or 512 columns gained nothing.
template <int RB, int MB, bool TURNED>
__global__ __launch_bounds__(256, RB <= 4 ? 2 : 1) void lora_narrow_kernel(LoraGroups g, const uint16_t* __restrict__ x,
                                                                           long long x_ld,
                                                                           const uint16_t* __restrict__ W, int r, int K,
                                                                           int slice, float* __restrict__ out) {
  constexpr int BM = 64 * MB, RP = 16 * RB, KT = 128;
  constexpr int LD = TURNED ? RP + 8 : KT + 8, STAGE = (TURNED ? KT : RP) * LD;
  __shared__ __attribute__((aligned(16))) uint16_t ws[2 * STAGE];
  __shared__ __attribute__((aligned(16))) uint16_t xs[4 * MB * 16 * KT];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row16 = lane & 15, q = lane >> 4;
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) lora_report(g);
  const LoraTile t = lora_tile(g, BM, blockIdx.x);
  if (t.e < 0) return;
  const int wave_row = 16 * MB * wave;
  const uint16_t* xr[MB][4];     // rows 4 i + q of each 16
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = wave_row + 16 * m + 4 * i + q;
      const int row = lora_row(g, t.row + at, at < t.rows);
      xr[m][i] = x + (long long)max(row, 0) * x_ld;   // a row that is none: any, its sums are dropped
    }
  const uint16_t* We = W + (long long)t.e * r * K;
  const int k_begin = blockIdx.y * slice, k_end = min(K, k_begin + slice);   // multiples of 8
  // Every load is made, at a place that exists, and what lies past the slice is
  // replaced by zeros where it is used: a load that may be skipped keeps the
  // compiler from counting how many are on their way, and it waits for all.
  u32x4 wv[RB];
  const auto load_w = [&](int k0) {
#pragma unroll
    for (int c = 0; c < RB; ++c) {
      const int i = tid + 256 * c;
      if constexpr (TURNED) {
        const int row = i / (2 * RB), rc = 8 * (i - row * (2 * RB));
        wv[c] = *reinterpret_cast<const u32x4*>(We + (long long)min(k0 + row, k_end - 1) * r + min(rc, r - 8));
      } else {
        wv[c] = *reinterpret_cast<const u32x4*>(We + (long long)min(i >> 4, r - 1) * K + min(k0 + 8 * (i & 15), k_end - 8));
      }
    }
  };
  const auto store_w = [&](int stage, int k0) {
    uint16_t* d = ws + stage * STAGE;
#pragma unroll
    for (int c = 0; c < RB; ++c) {
      const int i = tid + 256 * c;
      if constexpr (TURNED) {
        const int row = i / (2 * RB), rc = 8 * (i - row * (2 * RB));
        *reinterpret_cast<u32x4*>(d + row * LD + rc) = k0 + row < k_end ? wv[c] : u32x4{0, 0, 0, 0};
      } else {
        *reinterpret_cast<u32x4*>(d + (i >> 4) * LD + 8 * (i & 15)) = k0 + 8 * (i & 15) < k_end ? wv[c] : u32x4{0, 0, 0, 0};
      }
    }
  };
  const auto load_x = [&](int k0, u32x4 (&v)[MB][4]) {
    const int k = min(k0 + 8 * row16, k_end - 8);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[m][i] = *reinterpret_cast<const u32x4*>(xr[m][i] + k);
  };
  u32x4 xa[MB][4], xb[MB][4];
  f32x4 acc[MB][RB] = {};
  uint16_t* mine = xs + wave * (MB * 16 * KT);
  const int read16 = hidden(row16);
  // 16-byte piece c of row i of a wave's LDS lies at place c ^ i
  const auto compute = [&](int stage, int k0, const u32x4 (&v)[MB][4]) {
    const bool in = k0 + 8 * row16 < k_end;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + q;
        *reinterpret_cast<u32x4*>(mine + (16 * m + row) * KT + 8 * (row16 ^ row)) = in ? v[m][i] : u32x4{0, 0, 0, 0};
      }
    const uint16_t* d = ws + stage * STAGE;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 xf[MB];
#pragma unroll
      for (int m = 0; m < MB; ++m) xf[m] = load8(mine + (16 * m + read16) * KT + 8 * ((4 * j + q) ^ read16));
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        bf16x8 wf;
        if constexpr (TURNED) {
          const uint16_t* p = d + (32 * j + 8 * q + (row16 >> 2)) * LD + 16 * b + 4 * (row16 & 3);
          wf = read_crosswise(p, p + 4 * LD);
        } else {
          wf = load8(d + (16 * b + row16) * LD + 32 * j + 8 * q);
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[m][b] = mfma16(wf, xf[m], acc[m][b]);
      }
    }
  };
  // a step, while the next one's x and the weights after it are on their way; true:
  // it was the last
  const auto step = [&](int stage, int k0, const u32x4 (&v)[MB][4], u32x4 (&next)[MB][4]) {
    __syncthreads();
    store_w(stage ^ 1, k0 + KT);
    load_w(k0 + 2 * KT);
    load_x(k0 + KT, next);
    compute(stage, k0, v);
    return k0 + KT >= k_end;                     // the same for the whole workgroup
  };
  load_w(k_begin);
  load_x(k_begin, xa);
  store_w(0, k_begin);
  load_w(k_begin + KT);
  for (int k0 = k_begin;; k0 += 2 * KT) {
    if (step(0, k0, xa, xb)) break;
    if (step(1, k0 + KT, xb, xa)) break;
  }
  float* o = out + (long long)blockIdx.y * g.M_cap * r;
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int at = wave_row + 16 * m + row16;
    if (at >= t.rows) continue;
    const bool there = lora_row(g, t.row + at, true) >= 0;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int c = 16 * b + 4 * q;               // r is a multiple of 8: all four or none
      if (c < r)
        *reinterpret_cast<f32x4*>(o + (long long)(t.row + at) * r + c) = there ? acc[m][b] : f32x4{0, 0, 0, 0};
    }
  }
}

// The u of a row from value c (of 8) of its two parts, as a fragment: the slices'
// sums added in order, times s; the nearest bf16 value for c < r, what is left for c <
// 2 r, else 0.  Two parts hold u to 2^-17 of its value, far below the rounding of y.
// out (nullable): where the sum itself goes.
__device__ __forceinline__ bf16x8 u_fragment(const float* u, long long slice_len, int slices, int r, int c, float s,
                                             bool inside, float* out) {
  f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
  if (inside && c < 2 * r) {
    const int at = c < r ? c : c - r;
    const float* p = u + at;
    int i = 0;
    for (; i + 4 <= slices; i += 4) {
      f32x4 a[4], b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = *reinterpret_cast<const f32x4*>(p + (i + k) * slice_len);
        b[k] = *reinterpret_cast<const f32x4*>(p + (i + k) * slice_len + 4);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        lo += a[k];
        hi += b[k];
      }
    }
    for (; i < slices; ++i) {
      lo += *reinterpret_cast<const f32x4*>(p + i * slice_len);
      hi += *reinterpret_cast<const f32x4*>(p + i * slice_len + 4);
    }
    if (out && c < r) {
      *reinterpret_cast<f32x4*>(out + at) = lo;
      *reinterpret_cast<f32x4*>(out + at + 4) = hi;
    }
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = s * (i < 4 ? lo[i] : hi[i - 4]);
  u32x4 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const TwoParts p = two_parts(v[2 * i], v[2 * i + 1]);
    f[i] = c < r ? p.first : p.rest;
  }
  if (c >= 2 * r) f = u32x4{0, 0, 0, 0};          // (an infinite s)
  return __builtin_bit_cast(bf16x8, f);
}
// Eight sums and eight bf16 values of base, rounded once.
__device__ __forceinline__ u32x4 add_base(const float* v, u32x4 base) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack_bf16x2(v[2 * i] + __uint_as_float(base[i] << 16), v[2 * i + 1] + __uint_as_float(base[i] & 0xFFFF0000u));
  return o;
}
__device__ __forceinline__ uint32_t pick16(uint32_t lo, uint32_t hi, bool upper) {
  return __builtin_amdgcn_perm(hi, lo, upper ? 0x07060302u : 0x05040100u);
}

// ---------------------------------------------------------------- y = base + s u W^T
// A tile of 64 rows and a slice of N per workgroup, 128 columns at a time, the next
// step's base and the weights after it in flight.  A wave holds its 16 rows' u as
// two bf16 parts, [nearest r | rest r | zeros], one reduction of KS MFMA steps against
// the weights taken twice.  The weights come through LDS (two
// stages) as [column][r], W [N][r] as it is or with TURNED [r][N] (the backward's dx
// = w A) taken apart by byte permutations.  Column 8 i + j of a step lies in row 16
// j + i of LDS: MFMA j then gives a lane column j of its eight, so that 16 lanes
// load and store 256 bytes of a row.
//
// Measured: 14746 rows, r 64, N 4096 54 us, 4.4 TB/s; 16384 rows in 32 groups, r 32, N 7168
// (dx) 103 us, 4.5 TB/s; 8191 rows, r 16, N 5760 39 us, 4.8 TB/s; 8192 rows, r 128, N 7168
// 94 us, 2.5 TB/s: a weight fragment is read from LDS for 16 rows a wave, and again for the
// second part of u.  Tiles of 32 rows per wave spill at r 128; the weights turned by a kernel
// of their own cost 9 us more than they save.
template <int KS, bool TURNED>
__global__ __launch_bounds__(256, KS <= 4 ? 3 : 2) void lora_wide_kernel(LoraGroups g, const float* __restrict__ u_in,
                                                                         int slices, float* __restrict__ u_out,
                                                                         const uint16_t* __restrict__ W,
                                                                         const float* __restrict__ scale, int r, int N,
                                                                         int slice, const uint16_t* base, uint16_t* y,
                                                                         long long y_ld) {
  constexpr int BM = 64, RP = 16 * KS, NT = 128, LD = RP + 8, STAGE = NT * LD;
  __shared__ __attribute__((aligned(16))) uint16_t ws[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row16 = lane & 15, q = lane >> 4;
  const LoraTile t = lora_tile(g, BM, blockIdx.x);
  if (t.e < 0) return;
  const uint16_t* We = W + (long long)t.e * N * r;
  const int n_begin = blockIdx.y * slice, n_end = min(N, n_begin + slice);
  // TURNED: a thread takes eight columns of a pair of weight rows, KS / 2 times (KS
  // = 1: half of the threads, once)
  constexpr int NW = TURNED ? (KS == 1 ? 2 : KS) : KS;
  u32x4 wv[NW];
  const auto load_w = [&](int n0) {             // as in the narrow kernel: every load is made
#pragma unroll
    for (int c = 0; c < NW; ++c) {
      if constexpr (TURNED) {
        const int i = tid + 256 * (c / 2), row = 2 * (i >> 4) + (c & 1);
        wv[c] = *reinterpret_cast<const u32x4*>(We + (long long)min(row, r - 1) * N + min(n0 + 8 * (i & 15), n_end - 8));
      } else {
        const int i = tid + 256 * c, row = i / (2 * KS), rc = 8 * (i - row * (2 * KS));
        wv[c] = *reinterpret_cast<const u32x4*>(We + (long long)min(n0 + row, n_end - 1) * r + min(rc, r - 8));
      }
    }
  };
  const auto store_w = [&](int stage) {
    uint16_t* d = ws + stage * STAGE;
    if constexpr (TURNED) {
#pragma unroll
      for (int c = 0; c < NW; c += 2) {
        const int i = tid + 256 * (c / 2), row = 2 * (i >> 4);
        if (row < RP)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint32_t*>(d + (16 * j + (i & 15)) * LD + row) =
                pick16(wv[c][j / 2], wv[c + 1][j / 2], j & 1);
      }
    } else {
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        const int i = tid + 256 * c, row = i / (2 * KS), rc = 8 * (i - row * (2 * KS));
        *reinterpret_cast<u32x4*>(d + (16 * (row & 7) + (row >> 3)) * LD + rc) = wv[c];
      }
    }
  };
  load_w(n_begin);
  const int wave_row = 16 * wave;
  long long yo[4];             // rows 4 q + i of the wave's; -1: none
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = wave_row + 4 * q + i;
    const int row = lora_row(g, t.row + at, at < t.rows);
    yo[i] = row >= 0 ? (long long)row * y_ld : -1;
  }
  const uint16_t* from_base = base ? base : y;  // without a base: read, not used
  const auto load_base = [&](int n0, u32x4 (&v)[4]) {
    const int n = min(n0 + 8 * row16, n_end - 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const u32x4*>(from_base + max(yo[i], 0LL) + n);
  };
  u32x4 ba[4], bb[4];
  load_base(n_begin, ba);
  const float s = scale ? scale[t.e] : 1.0f;
  // the slices' sums of the tile, a thread taking every 256th four of its values, through
  // LDS: each wave adding up its own fragments reads everything twice, in KS loops one
  // after the other (3.3 times the kernel's time at 2048 rows, r 64 and 23 slices)
  bf16x8 uv[KS];
  {
    float* us = reinterpret_cast<float*>(ws);
    constexpr int ULD = RP + 4, AT_ONCE = KS >= 8 ? 1 : 8 / KS;
    const long long len = (long long)g.M_cap * r;
    const float* p = u_in + (long long)t.row * r;
    const int n = t.rows * r;                    // >= 8
    int at[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) at[k] = min(4 * (tid + 256 * k), n - 4);
    f32x4 v[KS] = {};
    int i = 0;
    for (; i + AT_ONCE <= slices; i += AT_ONCE) {
      f32x4 w[AT_ONCE][KS];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
#pragma unroll
        for (int k = 0; k < KS; ++k) w[j][k] = *reinterpret_cast<const f32x4*>(p + (i + j) * len + at[k]);
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
#pragma unroll
        for (int k = 0; k < KS; ++k) v[k] += w[j][k];
    }
    for (; i < slices; ++i)
#pragma unroll
      for (int k = 0; k < KS; ++k) v[k] += *reinterpret_cast<const f32x4*>(p + i * len + at[k]);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int row = at[k] / r;
      if (4 * (tid + 256 * k) < n) {
        *reinterpret_cast<f32x4*>(us + row * ULD + (at[k] - row * r)) = v[k];
        if (u_out && blockIdx.y == 0) *reinterpret_cast<f32x4*>(u_out + (long long)t.row * r + at[k]) = v[k];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KS; ++k)
      uv[k] = u_fragment(us + (wave_row + row16) * ULD, 0, 1, r, 8 * (4 * k + q), s, wave_row + row16 < t.rows, nullptr);
    __syncthreads();
  }
  int from[KS];           // this lane's place in a weight row at each step; -1: past both parts
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const int c = 8 * (4 * k + q);
    from[k] = c < r ? c : c < 2 * r ? c - r : -1;
  }
  const auto compute = [&](int stage, int n0, const u32x4 (&v)[4]) {
    const uint16_t* d = ws + stage * STAGE + row16 * LD;
    f32x4 acc[8] = {};
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bf16x8 wf = from[k] >= 0 ? load8(d + 16 * j * LD + from[k]) : zero8();
        acc[j] = mfma16(uv[k], wf, acc[j]);
      }
    const bool in = n0 + 8 * row16 < n_end;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = acc[j][i];
      const u32x4 out = add_base(o, base ? v[i] : u32x4{0, 0, 0, 0});
      if (in && yo[i] >= 0) *reinterpret_cast<u32x4*>(y + yo[i] + n0 + 8 * row16) = out;
    }
  };
  // a step, while the next one's base and the weights after it are on their way; true:
  // it was the last
  const auto step = [&](int stage, int n0, const u32x4 (&v)[4], u32x4 (&next)[4]) {
    __syncthreads();
    store_w(stage ^ 1);
    load_w(n0 + 2 * NT);
    load_base(n0 + NT, next);
    compute(stage, n0, v);
    return n0 + NT >= n_end;                      // the same for the whole workgroup
  };
  store_w(0);
  load_w(n_begin + NT);
  for (int n0 = n_begin;; n0 += 2 * NT) {
    if (step(0, n0, ba, bb)) break;
    if (step(1, n0 + NT, bb, ba)) break;
  }
}

// ---------------------------------------------------------------- few rows
// The same two products for a decoding batch, where what counts is how soon every
// weight is on its way: tiles of 16 rows whose operands go straight from memory to
// the MFMA.  The narrow one: 512 columns of K per workgroup, whose four waves' sums
// meet in LDS.  Measured: 1 row, r 16, K 7168, N 4096 3.6 and 5.1 us for the wide one,
// beside 3.2 us of the host for each launch; 64 rows in 32 groups 8.3 and 27.8 us at r 64,
// 14.6 and 59.2 at r 128, where each wave of the wide one adds up all 14 slices of u for
// itself.
template <int RB>
__global__ __launch_bounds__(256) void lora_few_narrow_kernel(LoraGroups g, const uint16_t* __restrict__ x,
                                                              long long x_ld, const uint16_t* __restrict__ A, int r,
                                                              int K, float* __restrict__ out) {
  constexpr int RP = 16 * RB, LD = RP + 4;
  __shared__ __attribute__((aligned(16))) float red[4 * 16 * LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row16 = lane & 15, q = lane >> 4;
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) lora_report(g);
  const LoraTile t = lora_tile(g, 16, blockIdx.x);
  if (t.e < 0) return;
  const int k0 = 512 * blockIdx.y + 128 * wave + 8 * q;
  bf16x8 av[4][RB], xv[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int k = k0 + 32 * j;
      av[j][b] = k < K ? load8(A + ((long long)t.e * r + min(16 * b + row16, r - 1)) * K + k) : zero8();
    }
  const int row = lora_row(g, t.row + row16, row16 < t.rows);
  const uint16_t* xr = x + (long long)max(row, 0) * x_ld;
#pragma unroll
  for (int j = 0; j < 4; ++j) xv[j] = k0 + 32 * j < K ? load8(xr + k0 + 32 * j) : zero8();
  f32x4 acc[RB] = {};
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = mfma16(av[j][b], xv[j], acc[b]);
  if (row < 0)
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int b = 0; b < RB; ++b) *reinterpret_cast<f32x4*>(&red[(wave * 16 + row16) * LD + 16 * b + 4 * q]) = acc[b];
  __syncthreads();
  float* o = out + ((long long)blockIdx.y * g.M_cap + t.row) * r;
  const int quads = r / 4;
  for (int i = tid; i < t.rows * quads; i += 256) {
    const int at = i / quads, c = 4 * (i - at * quads);
    f32x4 v = *reinterpret_cast<const f32x4*>(&red[at * LD + c]);
#pragma unroll
    for (int w = 1; w < 4; ++w) v += *reinterpret_cast<const f32x4*>(&red[(w * 16 + at) * LD + c]);
    *reinterpret_cast<f32x4*>(o + (long long)at * r + c) = v;
  }
}

// The wide one: NB times 32 columns of y per wave; the rows of two MFMAs are chosen
// so that a lane's eight products are eight consecutive columns.
template <int KS, int NB>
__global__ __launch_bounds__(256) void lora_few_wide_kernel(LoraGroups g, const float* __restrict__ u_in, int slices,
                                                            float* __restrict__ u_out, const uint16_t* __restrict__ B,
                                                            const float* __restrict__ scale, int r, int N,
                                                            const uint16_t* base, uint16_t* y, long long y_ld) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row16 = lane & 15, q = lane >> 4;
  const LoraTile t = lora_tile(g, 16, blockIdx.x);
  const int n0 = 32 * NB * (4 * blockIdx.y + wave);
  if (t.e < 0 || n0 >= N) return;
  const float s = scale ? scale[t.e] : 1.0f;
  bf16x8 bv[NB][KS][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int c = 8 * (4 * k + q);
      const int from = c < r ? c : c < 2 * r ? c - r : -1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = min(n0 + 32 * b + 8 * (row16 >> 2) + (row16 & 3) + 4 * j, N - 1);
        const bf16x8 v = load8(B + ((long long)t.e * N + n) * r + max(from, 0));
        bv[b][k][j] = from >= 0 ? v : zero8();
      }
    }
  const int row = lora_row(g, t.row + row16, row16 < t.rows);
  const long long yo = (long long)max(row, 0) * y_ld;
  u32x4 old[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int n = n0 + 32 * b + 8 * q;
    old[b] = u32x4{0, 0, 0, 0};
    if (base && row >= 0 && n < N) old[b] = *reinterpret_cast<const u32x4*>(base + yo + n);
  }
  f32x4 acc[NB][2] = {};
  const long long p = (long long)(t.row + row16) * r;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const bf16x8 uv = u_fragment(u_in + p, (long long)g.M_cap * r, slices, r, 8 * (4 * k + q), s, row16 < t.rows,
                                 u_out && blockIdx.y == 0 && wave == 0 ? u_out + p : nullptr);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[b][j] = mfma16(bv[b][k][j], uv, acc[b][j]);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int n = n0 + 32 * b + 8 * q;
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = acc[b][i >> 2][i & 3];
    if (row >= 0 && n < N) *reinterpret_cast<u32x4*>(y + yo + n) = add_base(o, old[b]);
  }
}

// Both products in one launch where an adapter's A is small: each workgroup of a
// tile computes the whole u (its eight waves take runs of 64 columns of K in turn,
// AT_ONCE of them on their way), then a slice of y's columns, NB runs of 32 at a time
// for each wave.  With TURNED both weights lie the other way round (the backward's w and
// dx) and are read crosswise from LDS.  Measured under the profiler: 58 rows in 32 groups, r
// 16, K 2880, N 5760 7.4 us for 10.5 MB, 1 row, K 7168, N 4096 8.4 (calls one after the other
// 6.7 and 7.7): the products one after the other, each a few trips to memory of 0.7 us.  A's
// loads wait for src, though they do not need it, and a run's for the one before.  Calls when
// it was tuned: A and x loaded as the MFMA takes them 9.6; one, three or more runs at once 8.4
// to 9.0 at NB 1 for 8.1; y's columns one run at a time 8.0.
template <int RB, int AT_ONCE, int NB, bool TURNED>
__global__ __launch_bounds__(512) void lora_few_kernel(LoraGroups g, const uint16_t* __restrict__ x, long long x_ld,
                                                       const uint16_t* __restrict__ A, const uint16_t* __restrict__ B,
                                                       const float* __restrict__ scale, int r, int K, int N, int slice,
                                                       const uint16_t* base, uint16_t* y, long long y_ld,
                                                       float* __restrict__ u_out) {
  constexpr int RP = 16 * RB, LD = RP + 4, WAVES = 8;
  // a wave's piece of LDS: 64 columns of x's 16 rows, then what it needs of the weights
  // (the first ones of 64 columns, 16 ranks or with TURNED all; with TURNED the second ones
  // of 32 columns, from the start)
  constexpr int XLD = 64 + 8, ROWS = 16 * XLD, WLD = RP + 8, BLD = 32 + 8;
  constexpr int MINE = ROWS + (TURNED ? 64 * WLD : ROWS);
  __shared__ __attribute__((aligned(16))) float red[WAVES * 16 * LD];
  __shared__ __attribute__((aligned(16))) uint16_t xs[WAVES * MINE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row16 = lane & 15, q = lane >> 4;
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) lora_report(g);
  const LoraTile t = lora_tile(g, 16, blockIdx.x);
  if (t.e < 0) return;
  const int n_end = min(N, (int)(blockIdx.y + 1) * slice);
  int n0 = blockIdx.y * slice + 32 * wave;
  int from[RB];
#pragma unroll
  for (int k = 0; k < RB; ++k) {
    const int c = 8 * (4 * k + q);
    from[k] = c < r ? c : c < 2 * r ? c - r : -1;
  }
  // as they lie in memory: fragments, or with TURNED rows of 32 columns, 16 a load
  u32x4 bv[NB][TURNED ? RB : 2 * RB];
  const auto load_b = [&]() {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int k = 0; k < RB; ++k) {
        const int first = n0 + 32 * WAVES * b;
        if constexpr (TURNED) {
          const uint16_t* row = B + ((long long)t.e * r + min(16 * k + (lane >> 2), r - 1)) * N;
          bv[b][k] = *reinterpret_cast<const u32x4*>(row + min(first + 8 * (lane & 3), N - 8));
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int n = min(first + 8 * (row16 >> 2) + (row16 & 3) + 4 * j, N - 1);
            bv[b][2 * k + j] = *reinterpret_cast<const u32x4*>(B + ((long long)t.e * N + n) * r + max(from[k], 0));
          }
        }
      }
  };
  load_b();
  const uint16_t* Ae = A + (long long)t.e * r * K;
  const float s = scale ? scale[t.e] : 1.0f;
  const int row = lora_row(g, t.row + row16, row16 < t.rows);
  // eight lanes load 128 bytes of a row: the MFMA's operands, of which neighbouring lanes
  // hold different rows, come through LDS (read from memory, each of them visits 64 lines)
  const int sub = lane >> 3, piece = lane & 7;
  const uint16_t* xr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) xr[i] = x + (long long)max(__shfl(row, 8 * i + sub, 64), 0) * x_ld;
  uint16_t* mine = xs + wave * MINE;
  const int read16 = hidden(row16);
  const long long yo = (long long)max(row, 0) * y_ld;
  u32x4 old[NB] = {};
  const auto load_base = [&]() {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int n = n0 + 32 * WAVES * b + 8 * q;
      if (base && row >= 0 && n < n_end) old[b] = *reinterpret_cast<const u32x4*>(base + yo + n);
    }
  };
  load_base();
  f32x4 acc[RB] = {};
  for (int k0 = 64 * wave; k0 < K; k0 += 64 * WAVES * AT_ONCE) {
    u32x4 av[AT_ONCE][2 * RB], xv[AT_ONCE][2];
#pragma unroll
    for (int n = 0; n < AT_ONCE; ++n) {
      const int first = k0 + 64 * WAVES * n, c = min(first + 8 * piece, K - 8);
#pragma unroll
      for (int i = 0; i < 2 * RB; ++i) {
        if constexpr (TURNED) {
          const int at = lane + 64 * i, col = at / (2 * RB), rc = 8 * (at - col * (2 * RB));
          av[n][i] = *reinterpret_cast<const u32x4*>(Ae + (long long)min(first + col, K - 1) * r + min(rc, r - 8));
        } else {
          av[n][i] = *reinterpret_cast<const u32x4*>(Ae + (long long)min(8 * i + sub, r - 1) * K + c);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) xv[n][i] = *reinterpret_cast<const u32x4*>(xr[i] + c);
    }
#pragma unroll
    for (int n = 0; n < AT_ONCE; ++n) {
      const int first = k0 + 64 * WAVES * n;
      const u32x4 none = {0, 0, 0, 0};
      const auto through = [&](uint16_t* lds, const u32x4& v0, const u32x4& v1, bf16x8 (&f)[2]) {
        const bool in = first + 8 * piece < K;
        *reinterpret_cast<u32x4*>(lds + sub * XLD + 8 * piece) = in ? v0 : none;
        *reinterpret_cast<u32x4*>(lds + (8 + sub) * XLD + 8 * piece) = in ? v1 : none;
#pragma unroll
        for (int j = 0; j < 2; ++j) f[j] = load8(lds + read16 * XLD + 8 * (4 * j + q));
      };
      bf16x8 xf[2];
      through(mine, xv[n][0], xv[n][1], xf);
      if constexpr (TURNED) {
#pragma unroll
        for (int i = 0; i < 2 * RB; ++i) {
          const int at = lane + 64 * i, col = at / (2 * RB), rc = 8 * (at - col * (2 * RB));
          *reinterpret_cast<u32x4*>(mine + ROWS + col * WLD + rc) = first + col < K ? av[n][i] : none;
        }
      }
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        bf16x8 af[2];
        if constexpr (TURNED) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint16_t* p = mine + ROWS + (32 * j + 8 * q + (read16 >> 2)) * WLD + 16 * b + 4 * (read16 & 3);
            af[j] = read_crosswise(p, p + 4 * WLD);
          }
        } else {
          through(mine + ROWS, av[n][2 * b], av[n][2 * b + 1], af);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[b] = mfma16(af[j], xf[j], acc[b]);
      }
    }
  }
  if (row < 0)
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int b = 0; b < RB; ++b) *reinterpret_cast<f32x4*>(&red[(wave * 16 + row16) * LD + 16 * b + 4 * q]) = acc[b];
  __syncthreads();
  // the waves' sums, in the place of the first one's
  const int quads = r / 4;
  for (int i = tid; i < 16 * quads; i += 512) {
    const int at = i / quads, c = 4 * (i - at * quads);
    f32x4 v = *reinterpret_cast<const f32x4*>(&red[at * LD + c]);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += *reinterpret_cast<const f32x4*>(&red[(w * 16 + at) * LD + c]);
    *reinterpret_cast<f32x4*>(&red[at * LD + c]) = v;
    if (u_out && blockIdx.y == 0 && at < t.rows) *reinterpret_cast<f32x4*>(u_out + (long long)(t.row + at) * r + c) = v;
  }
  __syncthreads();
  bf16x8 uv[RB];
#pragma unroll
  for (int k = 0; k < RB; ++k) uv[k] = u_fragment(&red[row16 * LD], 0, 1, r, 8 * (4 * k + q), s, true, nullptr);
  while (n0 < n_end) {
    u32x4 w[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      f32x4 out[2] = {};
      if constexpr (TURNED)
#pragma unroll
        for (int k = 0; k < RB; ++k)
          *reinterpret_cast<u32x4*>(mine + (16 * k + (lane >> 2)) * BLD + 8 * (lane & 3)) = bv[b][k];
#pragma unroll
      for (int k = 0; k < RB; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          bf16x8 bf;
          if constexpr (TURNED) {
            const uint16_t* p = mine + (max(from[k], 0) + (read16 >> 2)) * BLD + 8 * (read16 & 3) + 4 * j;
            bf = read_crosswise(p, p + 4 * BLD);
          } else {
            bf = __builtin_bit_cast(bf16x8, bv[b][2 * k + j]);
          }
          out[j] = mfma16(from[k] >= 0 ? bf : zero8(), uv[k], out[j]);
        }
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = out[i >> 2][i & 3];
      w[b] = add_base(o, old[b]);
    }
    const int n1 = n0 + 8 * q;
    n0 += 32 * WAVES * NB;
    if (n0 < n_end) {
      load_b();
      load_base();
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int n = n1 + 32 * WAVES * b;
      if (row >= 0 && n < n_end) *reinterpret_cast<u32x4*>(y + yo + n) = w[b];
    }
  }
}

// ---------------------------------------------------------------- dA, dB
// The sums over a group's rows of (s u_i) v_i^T, u fp32 [M_cap][r], v bf16 rows of
// C columns: dA from w and x, dB from u and dy.  A piece of a group's rows and 64 CW
// columns per workgroup, 16 CW for each wave, 32 rows at a time, the next ones on their
// way.  The MFMA wants eight rows of one column per lane where memory has columns side
// by side: a wave puts its rows into a piece of LDS of its own and reads them crosswise.
// u goes in as three bf16 parts, 24 bits of it, so that the sums are those of fp32
// products; the parts of 32 rows are made once for the four waves, in LDS (two stages).
// The operand that comes first gives a lane four consecutive places of the product: the
// columns for [r][C], the ranks for [C][r].
//
// Measured (K 7168, N 4096): 8191 rows, r 16, K 2880, N 5760 30 us, 4.8 TB/s; 16384 rows in
// 32 groups, r 32 126 us, 2.9 TB/s beside 235 MB of dx that go to memory meanwhile; 14746
// rows, r 64 117 us, 2.8 TB/s; 8192 rows, r 128, K and N 7168 155 us, 1.5 TB/s: every column
// block reads u and makes its parts again.  With the rows in registers, taken apart there,
// r 32 took 119 and r 16 28, but r 64 178 for 120 and r 128 197 for 152.  dB in the pass that
// makes w (dy read once, two barriers a step): all of the backward 263 for 279 us at r 32, 85
// for 83 at r 16, 271 for 264 at r 64.
struct LoraSum {
  const float* u;
  const uint16_t* v;
  long long v_ld;
  int C;
  float* out;        // [L][r][C], or [L][C][r] for dB
  float* part;       // [slots][r][C] likewise, of groups of more than one piece
};
constexpr int kLoraPiece = 1024;   // rows of a piece, at most

// The parts of u: rank k of one of them holds 32 rows, 16-byte piece c at c ^ (k / 4).
__device__ __forceinline__ int lora_part(int k, int c) { return 32 * k + 8 * (c ^ (k >> 2 & 3)); }

template <int RB, int CW>
struct LoraSumLds {
  static constexpr int XLD = 16 * CW + 16;       // four rows of 32 bytes, read crosswise, in different banks
  int rows[kLoraPiece + 32];
  alignas(16) uint16_t us[2 * 3 * 16 * RB * 32], xs[4 * 32 * XLD];
};
template <int RB, int CW, bool TURNED>
__device__ __forceinline__ void lora_sum(const LoraTile& t, const LoraGroups& g, const LoraSum& p, int block, float s, int r,
                                         int accumulate, LoraSumLds<RB, CW>& lds) {
  constexpr int RP = 16 * RB, PART = RP * 32, STAGE = 3 * PART, XLD = LoraSumLds<RB, CW>::XLD;
  constexpr int KT = 16 * CW, PIECES = KT / 8, RL = 64 / PIECES, NL = 32 / RL;   // RL rows a load, NL loads
  int* rows = lds.rows;
  uint16_t *us = lds.us, *xs = lds.xs;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row16 = lane & 15, q = lane >> 4;
  const int C = p.C, c0 = block * (4 * KT) + KT * wave;
  for (int i = tid; i < t.rows + 32; i += 256) rows[i] = lora_row(g, t.row + i, i < t.rows);
  __syncthreads();
  // thread: value ri of row pairs
  const int ri = tid % RP, pair0 = tid / RP;
  float uv[RB][2];
  const auto load_u = [&](int i0) {              // as in the narrow kernel: every load is made
#pragma unroll
    for (int k = 0; k < RB; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = min(i0 + 2 * (pair0 + k * (256 / RP)) + h, t.rows - 1);
        uv[k][h] = p.u[(long long)(t.row + at) * r + min(ri, r - 1)];
      }
  };
  const auto store_u = [&](int stage, int i0) {
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      const int pair = pair0 + k * (256 / RP), at = i0 + 2 * pair;
      const float v0 = rows[at] >= 0 ? s * uv[k][0] : 0.0f, v1 = rows[at + 1] >= 0 ? s * uv[k][1] : 0.0f;
      const float r0 = rest_of(v0), r1 = rest_of(v1);
      uint32_t* o = reinterpret_cast<uint32_t*>(us + stage * STAGE + lora_part(ri, pair >> 2)) + (pair & 3);
      o[0] = upper_half(v0) | upper_half(v1) << 16;
      o[PART / 2] = upper_half(r0) | upper_half(r1) << 16;
      o[PART] = pack_bf16x2(rest_of(r0), rest_of(r1));
    }
  };
  uint16_t* mine = xs + wave * (32 * XLD);
  const int read16 = hidden(row16);
  const int sub = lane / PIECES, piece = lane % PIECES;
  const uint16_t* vc = p.v + min(c0 + 8 * piece, C - 8);
  const auto load_v = [&](int i0, u32x4 (&v)[NL]) {   // (columns past the last one: their sums are dropped)
#pragma unroll
    for (int i = 0; i < NL; ++i)
      v[i] = *reinterpret_cast<const u32x4*>(vc + (long long)max(rows[min(i0, t.rows - 1) + RL * i + sub], 0) * p.v_ld);
  };
  const auto store_v = [&](int i0, const u32x4 (&v)[NL]) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int row = RL * i + sub;
      *reinterpret_cast<u32x4*>(mine + row * XLD + 8 * piece) = rows[i0 + row] >= 0 ? v[i] : u32x4{0, 0, 0, 0};
    }
  };
  f32x4 acc[RB][CW] = {};
  const auto compute = [&](int stage) {
    const uint16_t* d = us + stage * STAGE + lora_part(row16, q);
    const uint16_t* c = mine + (8 * q + (read16 >> 2)) * XLD + 4 * (read16 & 3);
    const auto column = [&](int j) { return read_crosswise(c + 16 * j, c + 16 * j + 4 * XLD); };
    const auto part_of_u = [&](int k, int part) { return load8(d + part * PART + 16 * 32 * k); };
    // what fewer registers hold stays over the loop, the lowest parts come first
    if constexpr (RB <= 2) {
      bf16x8 uf[RB][3];
#pragma unroll
      for (int k = 0; k < RB; ++k)
#pragma unroll
        for (int part = 0; part < 3; ++part) uf[k][part] = part_of_u(k, part);
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        const bf16x8 col = column(j);
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
          for (int k = 0; k < RB; ++k)
            acc[k][j] = TURNED ? mfma16(uf[k][part], col, acc[k][j]) : mfma16(col, uf[k][part], acc[k][j]);
      }
    } else {
      bf16x8 col[CW];
#pragma unroll
      for (int j = 0; j < CW; ++j) col[j] = column(j);
#pragma unroll
      for (int k = 0; k < RB; ++k)
#pragma unroll
        for (int part = 2; part >= 0; --part) {
          const bf16x8 uf = part_of_u(k, part);
#pragma unroll
          for (int j = 0; j < CW; ++j)
            acc[k][j] = TURNED ? mfma16(uf, col[j], acc[k][j]) : mfma16(col[j], uf, acc[k][j]);
        }
    }
  };
  if (t.rows > 0) {
    u32x4 v[NL];
    load_u(0);
    load_v(0, v);
    store_u(0, 0);
    load_u(32);
    for (int i0 = 0, stage = 0;; i0 += 32, stage ^= 1) {
      store_v(i0, v);
      load_v(i0 + 32, v);                        // while these 32 rows are computed
      __syncthreads();
      if (i0 + 32 < t.rows) {
        store_u(stage ^ 1, i0 + 32);
        load_u(i0 + 64);
      }
      compute(stage);
      if (i0 + 32 >= t.rows) break;              // the same for the whole workgroup
    }
  }
  const bool whole = t.pieces == 1;
  float* o = whole ? p.out + (long long)t.e * r * C : p.part + (long long)t.slot * r * C;
  const bool add = whole && accumulate;
#pragma unroll
  for (int k = 0; k < RB; ++k)
#pragma unroll
    for (int j = 0; j < CW; ++j) {
      // (r and C are multiples of 8: all four or none)
      const int rk = 16 * k + (TURNED ? 4 * q : row16), c = c0 + 16 * j + (TURNED ? row16 : 4 * q);
      if (rk >= r || c >= C) continue;
      f32x4* d = reinterpret_cast<f32x4*>(o + (TURNED ? (long long)c * r + rk : (long long)rk * C + c));
      *d = add ? *d + acc[k][j] : acc[k][j];
    }
}
template <int RB, int CW>
__global__ __launch_bounds__(256, RB <= 2 ? 3 : 2) void lora_sum_kernel(LoraGroups g, LoraSum a, LoraSum b, int a_blocks,
                                                                        int blocks, const float* __restrict__ scale, int r,
                                                                        int piece, int accumulate) {
  __shared__ LoraSumLds<RB, CW> lds;
  // neighbouring workgroups take the columns of the same rows, so that whole rows are on
  // their way at once (with the pieces as neighbours r 16 takes 28 us for 29, but r 32 134
  // for 128, r 128 166 for 150)
  const int block = blockIdx.x % blocks;
  const LoraTile t = lora_piece(g, piece, accumulate ? 0 : 1, blockIdx.x / blocks);
  if (t.e < 0) return;
  const float s = scale ? scale[t.e] : 1.0f;
  if (block < a_blocks) lora_sum<RB, CW, false>(t, g, a, block, s, r, accumulate, lds);
  else lora_sum<RB, CW, true>(t, g, b, block - a_blocks, s, r, accumulate, lds);
}

// The pieces of the groups that have more than one, added in their order: a
// workgroup takes 1024 values of the blockIdx.y-th such group.
__global__ __launch_bounds__(256) void lora_join_kernel(LoraGroups g, LoraSum a, LoraSum b, int a_blocks, int r,
                                                        int piece, int accumulate) {
  const bool first = (int)blockIdx.x < a_blocks;
  const LoraTile t = lora_many(g, piece, blockIdx.y);
  if (t.e < 0) return;
  const LoraSum& p = first ? a : b;
  const long long size = (long long)r * p.C;
  const long long i = 4 * ((long long)(first ? blockIdx.x : blockIdx.x - a_blocks) * 256 + threadIdx.x);
  if (i >= size) return;
  const float* src = p.part + (long long)t.slot * size + i;
  f32x4 s = *reinterpret_cast<const f32x4*>(src);
  int k = 1;
  for (; k + 8 <= t.pieces; k += 8) {
    f32x4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const f32x4*>(src + (k + j) * size);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[j];
  }
  for (; k < t.pieces; ++k) s += *reinterpret_cast<const f32x4*>(src + k * size);
  f32x4* d = reinterpret_cast<f32x4*>(p.out + (long long)t.e * size + i);
  *d = accumulate ? *d + s : s;
}

// Zeros for the gradients of a call without rows.
__global__ __launch_bounds__(256) void lora_zero_kernel(float* p, long long n) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) p[i] = 0.0f;
}

}  // namespace moe
