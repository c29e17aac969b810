// MXFP4: OCP e2m1 codes in blocks of 32 values with one E8M0 scale, their
// quantisation and their grouped product on the block-scaled MFMA.
#pragma once

#include "group_gemm.hpp"
#include "operator_args.hpp"

namespace moe {

// Block-scale exponent for e2m1 elements (largest value 6 = 1.5 * 2^2): the
// smallest E with amax / 2^E <= 6, as mx_scale_exponent for e4m3 and e5m2.
__device__ __forceinline__ int mx4_scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax) & 0x7FFFFFFFu;
  if (u >= 0x7F800000u) return 128;
  const uint32_t ebits = u >> 23;
  if (ebits == 0) return -127;
  const int E = static_cast<int>(ebits) - 127 - 2 + ((u & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return E < -127 ? -127 : E;
}

// 2^E as fp32, E in [-127, 127] (2^-127 is a subnormal)
__device__ __forceinline__ float pow2f(int E) {
  return E == -127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(E + 127) << 23);
}

// Eight values -> eight e2m1 codes of v / 2^E (value i in bits 4 i .. + 3),
// round to nearest, ties to even (v_cvt_scalef32_pk_fp4_f32; equal to the
// exact rounding on every bf16 value up to 6 2^E in size, over the scales'
// whole range, checked on the GPU).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  return w;
}

// Routed rows: the sum of the clamped counts, at most M_cap, by one wave alone.
__device__ __forceinline__ int routed_rows(const int* __restrict__ counts, int E, int M_cap) {
  long long n = 0;
  for (int e = threadIdx.x & 63; e < E; e += 64) n += max(counts[e], 0);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d, 64);
  return (int)(n < M_cap ? n : M_cap);
}

// Row-wise quantisation of a bf16 [R][C] matrix: 4 lanes per 32-value block,
// 16 bytes read and 4 bytes of codes written per lane, U of them in flight.  A
// block holding a NaN or an infinity gets the NaN scale 0xFF and zero codes
// (e2m1 has no NaN).
template <int U>
__global__ __launch_bounds__(256) void mx4_rows_kernel(const uint16_t* __restrict__ v, int R, int C,
                                                       const int* __restrict__ counts, int E,
                                                       uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  const long long rows = counts ? routed_rows(counts, E, R) : R;
  const long long total = rows * (C >> 3);   // 16-byte chunks: a multiple of 4
  for (long long i0 = (long long)blockIdx.x * 256 * U + threadIdx.x; i0 < total;
       i0 += (long long)gridDim.x * 256 * U) {
    uint4 u[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      u[k] = make_uint4(0u, 0u, 0u, 0u);
      if (i0 + 256 * k < total) u[k] = reinterpret_cast<const uint4*>(v)[i0 + 256 * k];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long i = i0 + 256 * k;
      const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      // the block's largest magnitude as bits: bf16 bits order like the values,
      // and a NaN's are above infinity's
      uint32_t mag = 0;
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        mag = max(mag, max((w[j] << 16) & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
      }
      mag = max(mag, (uint32_t)__shfl_xor((int)mag, 1, 64));
      mag = max(mag, (uint32_t)__shfl_xor((int)mag, 2, 64));
      const int X = mx4_scale_exponent(__uint_as_float(mag));   // (128 from infinity up)
      if (i < total) {
        reinterpret_cast<uint32_t*>(q)[i] = X == 128 ? 0u : e2m1x8(x, pow2f(X));
        if ((i & 3) == 0) s[i >> 2] = e8m0_byte(X);
      }
    }
  }
}

// Quantisation of a [K][N] weight along K (transposing): thread (n, kb) reads
// 32 rows of column n (a wave reads 128-byte row pieces) and writes the block
// kb of row n.  Offline.
__global__ __launch_bounds__(256) void mx4_weight_kn_kernel(const uint16_t* __restrict__ src, int N, int K,
                                                            uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  const int n = blockIdx.x * 256 + threadIdx.x, kb = blockIdx.y, e = blockIdx.z;
  if (n >= N) return;
  const uint16_t* W = src + ((long long)e * K + kb * 32) * N + n;
  float x[4][8];
  float amax = 0.0f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float f = bf16_to_f32(W[(long long)i * N]);
    x[i >> 3][i & 7] = f;
    amax = fmaxf(amax, fabsf(f));
    nan = nan || f != f;
  }
  const int X = nan ? 128 : mx4_scale_exponent(amax);
  const float sc = X == 128 ? 1.0f : pow2f(X);
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (X != 128) w = make_uint4(e2m1x8(x[0], sc), e2m1x8(x[1], sc), e2m1x8(x[2], sc), e2m1x8(x[3], sc));
  const long long row = (long long)e * N + n;
  *reinterpret_cast<uint4*>(q + row * (K / 2) + kb * 16) = w;
  s[row * (K / 32) + kb] = e8m0_byte(X);
}

// ---------------------------------------------------------------- groups
// Row and m-tile prefixes of the device counts for tiles of BM rows: the part
// of GroupScan that these kernels need, at half its LDS.
struct RowScan {
  int row_off[kMaxExperts + 1];
  int tile_off[kMaxExperts + 1];
  long long wave_tmp[16];
};

// As build_group_scan: counts are clamped (a negative one to 0, rows past
// M_cap dropped); the writer workgroup stores the offsets and status bits.
template <int NT, int BM>
__device__ void build_row_scan(RowScan& rs, const int* __restrict__ counts, int E, int M_cap,
                               int* offsets_out, int* status_out, bool writer) {
  const int t = threadIdx.x;
  constexpr int PER = (kMaxExperts + NT - 1) / NT;
  int c[PER];
  long long sum = 0;
  int neg = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * PER + i;
    c[i] = e < E ? counts[e] : 0;
    if (c[i] < 0) { neg = 1; c[i] = 0; }
    sum += c[i];
  }
  const long long incl = block_incl_scan<NT, long long>(sum, rs.wave_tmp);
  long long run = incl - sum;
  int tiles = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * PER + i;
    const long long o0 = run < M_cap ? run : M_cap;
    run += c[i];
    const long long o1 = run < M_cap ? run : M_cap;
    if (e < E) rs.row_off[e] = (int)o0;
    c[i] = ((int)(o1 - o0) + BM - 1) / BM;
    tiles += c[i];
  }
  if (t == NT - 1) rs.row_off[E] = run < M_cap ? (int)run : M_cap;   // (threads past E add nothing)
  const bool over = run > M_cap;
  int trun = block_incl_scan<NT, int>(tiles, rs.wave_tmp) - tiles;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * PER + i;
    if (e < E) rs.tile_off[e] = trun;
    trun += c[i];
  }
  if (t == NT - 1) rs.tile_off[E] = trun;
  // (__syncthreads_or tells whether any is set, not which bits)
  const bool any_neg = __syncthreads_or(neg), any_over = __syncthreads_or(over);
  const int st = (any_neg ? 1 : 0) | (any_over ? 2 : 0);
  if (writer) {
    if (offsets_out)
      for (int e = t; e <= E; e += NT) offsets_out[e] = rs.row_off[e];
    if (status_out && t == 0 && st) atomicOr(status_out, st);
  }
}

typedef int i32x4 __attribute__((ext_vector_type(4)));

// The 16 bytes of an e2m1 fragment as an operand of the f8f6f4 MFMA, whose
// other 16 bytes the 4-bit format does not read.
__device__ __forceinline__ i32x8 mx4_frag(i32x4 v) {
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

// What the f8f6f4 MFMA's sums are worth, of random codes against sums in 64 bits:
// with two e2m1 operands an instruction's products are added to fp32's rounding
// (2.4e-8 of their sizes' sum).  With an e4m3 operand, products are cut off below
// the largest one: an instruction of 64 values is off by up to 2^-11.8 of its
// largest product (6.8e-5 of the sizes' sum), whatever the accumulator holds,
// whose addition is rounded as fp32's.  The other operand's format and the plain
// e4m3 MFMA make no difference, so no order of sums avoids it; bf16 products of the
// decoded values would, at half the MFMA's peak.  Of 16384 x 4096 outputs of 8-bit
// rows, K = 7168, 0.4% are not the nearest bf16; the MXFP8 products are the same in
// this.

// ---------------------------------------------------------------- few rows
// The tiles of BM rows of up to 64 experts, lane e holding expert e's: built
// and searched by each wave alone, without LDS or barriers.
struct WaveScan {
  int row0, rows, tile0, tiles;   // of this lane's expert
  int total;                      // tiles of all
};
template <int BM>
__device__ __forceinline__ WaveScan wave_scan(const int* __restrict__ counts, int E, int M_cap, int* offsets_out,
                                              int* status_out, bool writer) {
  const int lane = threadIdx.x & 63;
  const int c = lane < E ? counts[lane] : 0;
  const bool neg = __any(c < 0);
  long long run = max(c, 0);
  const long long own = run;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long long o = __shfl_up(run, d, 64);
    if (lane >= d) run += o;
  }
  const bool over = __shfl(run, 63, 64) > M_cap;
  WaveScan w;
  w.row0 = (int)(run - own < M_cap ? run - own : M_cap);
  const int end = (int)(run < M_cap ? run : M_cap);
  w.rows = end - w.row0;
  w.tiles = (w.rows + BM - 1) / BM;
  int t = w.tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(t, d, 64);
    if (lane >= d) t += o;
  }
  w.tile0 = t - w.tiles;
  w.total = __shfl(t, 63, 64);
  if (writer) {
    if (offsets_out) {
      if (lane < E) offsets_out[lane] = w.row0;
      if (lane == E - 1) offsets_out[E] = end;
    }
    const int st = (neg ? 1 : 0) | (over ? 2 : 0);
    if (status_out && lane == 0 && st) atomicOr(status_out, st);
  }
  return w;
}

// Grouped product straight from memory, for groups of few rows, where what
// counts is to stream the active experts' weights at the memory's rate: a wave
// takes 16 columns of a tile of up to 16 rows of one group and all of K, or a
// quarter of it (SPLIT: the workgroup's 4 waves take the same 16 columns and
// add their sums through LDS in wave order; for launches of few waves).  Lane
// (r, q) = (l % 16, l / 16) of v_mfma_scale_f32_16x16x128_f8f6f4 holds, of an
// e2m1 operand, row r's block q (16 bytes) with its scale; of an e4m3 operand,
// bytes 16 q .. + 15 of the step's first 64 values and of its second 64, and the
// scale of block q.  The result's lane holds columns 4 q .. + 3 of row r.  Groups
// of four steps (512 values) of both operands are loaded two ahead of the one
// that is multiplied: loads return in order, so rows fetched later than the
// weights would wait for the weights behind them.
template <bool A4, bool SMALL_E, bool SPLIT>
__global__ __launch_bounds__(256) void mx4_gemm_rows_kernel(Mx4Args p) {
  __shared__ std::conditional_t<SMALL_E, int, RowScan> gs;
  __shared__ f32x4 red[SPLIT ? 3 : 1][SPLIT ? 64 : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  WaveScan ws;
  int ntiles;
  if constexpr (SMALL_E) {
    ws = wave_scan<16>(p.counts, p.E, p.M_cap, p.offsets_out, p.status_out, blockIdx.x == 0 && wave == 0);
    ntiles = ws.total;
  } else {
    build_row_scan<256, 16>(gs, p.counts, p.E, p.M_cap, p.offsets_out, p.status_out, blockIdx.x == 0);
    ntiles = gs.tile_off[p.E];
  }
  ntiles = __builtin_amdgcn_readfirstlane(ntiles);
  const int nblk = p.K >> 5;
  const int ncb = SPLIT ? p.N >> 4 : p.N >> 6;   // column blocks: of 16 (all waves) or of 64
  const long long items = (long long)ntiles * ncb;
  const long long ldb = p.K >> 1, lda = A4 ? p.K >> 1 : p.K;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int tile = __builtin_amdgcn_readfirstlane((int)(it % ntiles));   // (a group's tiles side by side)
    const int cb = __builtin_amdgcn_readfirstlane((int)(it / ntiles));
    const int n0 = SPLIT ? cb * 16 : cb * 64 + wave * 16;
    int e, row0, rows;
    if constexpr (SMALL_E) {
      e = __builtin_ctzll(__ballot(tile >= ws.tile0 && tile < ws.tile0 + ws.tiles));
      const int local = tile - __builtin_amdgcn_readlane(ws.tile0, e);
      row0 = __builtin_amdgcn_readlane(ws.row0, e) + local * 16;
      rows = min(16, __builtin_amdgcn_readlane(ws.rows, e) - local * 16);
    } else {
      int lo = 0, hi = p.E;   // the last e with tile_off[e] <= tile
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (gs.tile_off[mid] <= tile) lo = mid; else hi = mid;
      }
      e = __builtin_amdgcn_readfirstlane(lo);
      row0 = __builtin_amdgcn_readfirstlane(gs.row_off[e] + (tile - gs.tile_off[e]) * 16);
      rows = min(16, __builtin_amdgcn_readfirstlane(gs.row_off[e + 1]) - row0);
    }
    const long long brow = (long long)e * p.N + n0 + r;
    const uint8_t* bq = p.B + brow * ldb + q * 16;
    const uint8_t* bs = p.b_scales + brow * nblk;
    // (the last row again behind the tile's end: its results there are not
    // stored)
    const long long arow = row0 + min(r, rows - 1);
    const uint8_t* aq = p.A + arow * lda + (A4 ? q * 16 : (q >> 1) * 32 + (q & 1) * 16);
    const uint8_t* as = p.a_scales + arow * nblk;
    constexpr int AST = A4 ? 16 : 32;   // bytes per block of a row
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto mfma = [&](i32x4 bv, int sb, i32x4 a0, i32x4 a1, int sa) {
      if constexpr (A4)
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx4_frag(bv), mx4_frag(a0), acc, 4, 4, 0, sb, 0, sa);
      else
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            mx4_frag(bv), __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7), acc, 4, 0, 0, sb, 0, sa);
    };
    // a group of 16 blocks (4 steps): the codes, and the 16 scales of each row,
    // byte 4 s + q of them this lane's
    struct Group { i32x4 b[4], a0[4], a1[A4 ? 1 : 4], sb, sa; };
    auto load = [&](int g) {
      Group v;
      const uint8_t* bp = bq + (long long)g * 256;
      const uint8_t* ap = aq + (long long)g * 16 * AST;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        v.b[s] = *reinterpret_cast<const i32x4*>(bp + 64 * s);
        v.a0[s] = *reinterpret_cast<const i32x4*>(ap + 4 * s * AST);
        if constexpr (!A4) v.a1[s] = *reinterpret_cast<const i32x4*>(ap + 4 * s * AST + 64);
      }
      __builtin_memcpy(&v.sb, bs + 16 * g, 16);
      __builtin_memcpy(&v.sa, as + 16 * g, 16);
      return v;
    };
    auto use = [&](const Group& v) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        mfma(v.b[s], (int)((uint32_t)v.sb[s] >> (8 * q)), v.a0[s], v.a1[A4 ? 0 : s], (int)((uint32_t)v.sa[s] >> (8 * q)));
    };
    const int ngrp = nblk >> 4;
    constexpr int ST = SPLIT ? 4 : 1;
    const int g0 = SPLIT ? wave : 0;
    // the blocks behind the last whole group first, so that their loads do not
    // stand alone at the end (SPLIT: the wave whose turn that group would be):
    // zero codes and scale 1 past the end of K, and the scales byte by byte,
    // since 16 bytes would leave the row
    Group t;
    const bool tail = nblk > 16 * ngrp && (!SPLIT || ngrp % 4 == wave);
    if (tail) {
      const i32x4 z = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int k0 = 16 * ngrp + 4 * s;
        const uint8_t* ap = aq + (long long)k0 * AST;
        const bool in = k0 + q < nblk;
        t.b[s] = in ? *reinterpret_cast<const i32x4*>(bq + (long long)k0 * 16) : z;
        t.a0[s] = (A4 ? in : k0 + (q >> 1) < nblk) ? *reinterpret_cast<const i32x4*>(ap) : z;
        if constexpr (!A4) t.a1[s] = k0 + 2 + (q >> 1) < nblk ? *reinterpret_cast<const i32x4*>(ap + 64) : z;
        t.sb[s] = in ? bs[k0 + q] : 127;
        t.sa[s] = in ? as[k0 + q] : 127;
      }
    }
    Group x, y;
    if (g0 < ngrp) {
      x = load(g0);
      y = load(min(g0 + ST, ngrp - 1));
    }
    if (tail) {
#pragma unroll
      for (int s = 0; s < 4; ++s) mfma(t.b[s], t.sb[s], t.a0[s], t.a1[A4 ? 0 : s], t.sa[s]);
    }
    if (g0 < ngrp) {
      int g = g0;
      for (; g + 2 * ST < ngrp; g += 2 * ST) {
        use(x);
        x = load(g + 2 * ST);
        use(y);
        y = load(min(g + 3 * ST, ngrp - 1));
      }
      use(x);
      if (g + ST < ngrp) use(y);
    }
    if constexpr (SPLIT) {
      __syncthreads();   // the previous item's sums are read
      if (wave > 0) red[wave - 1][lane] = acc;
      __syncthreads();
      if (wave > 0) continue;
      acc = acc + red[0][lane] + red[1][lane] + red[2][lane];
    }
    if (r < rows)
      *reinterpret_cast<uint2*>(p.C + (long long)(row0 + r) * p.N + n0 + 4 * q) =
          make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
  }
}

// ---------------------------------------------------------------- many rows
constexpr int MX4_BM = 256, MX4_BN = 256;

// Tile column (weight row) that row rho of a staged 32-row block holds.  The 32
// x 32 MFMA leaves lane half h with rows 8 a + 4 h .. + 3, a = 0 .. 3: dealt out
// in fours like this, half h holds 8 consecutive columns over a = 0, 1 and 8
// over a = 2, 3, each 16 bytes of bf16.
__device__ __forceinline__ int mx4_col(int rho) {
  return (rho & ~31) + 16 * ((rho >> 4) & 1) + 8 * ((rho >> 2) & 1) + 4 * ((rho >> 3) & 1) + (rho & 3);
}

// v_permlane16_swap: in each half of the wave, lanes 16..31 of x change places
// with lanes 0..15 of y.
__device__ __forceinline__ void swap16(uint32_t& x, uint32_t& y) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
  x = r[0];
  y = r[1];
}

// Staged weight rows of 64 bytes (4 chunks, 8-bit rows): row r's chunk c sits at
// c ^ (r / 4) % 4.  A 32 x 32 read's pass (16 lanes that agree in the chunk and
// in the parity of row bits 2..4) then takes each of the 16 bank groups once.
__device__ __forceinline__ int mx4_off64(int r, int c) { return r * 64 + ((c ^ ((r >> 2) & 3)) << 4); }

// Grouped product of e2m1 (A4) or e4m3 rows and e2m1 weights on 256 x 256
// tiles: 8 waves in a 4 x 2 grid of 64 x 128,
// v_mfma_scale_f32_32x32x64_f8f6f4.  A K-tile is 128 bytes of each row of A, 256
// e2m1 or 128 e4m3 values, and as many of B, staged by LDS-DMA in NST stages (2
// of 64 KB, or 3 of 48 KB).  The fragment reads are free of bank conflicts; the
// barrier that frees a stage sits before the last of a K-tile's k-steps (of 64
// values), whose fragments are in registers.  A block of 32 values is one
// 16-byte chunk of e2m1 codes or two of e4m3, so a K that ends inside a K-tile
// masks whole chunks: their DMA is sent out of the descriptor's range and reads
// zeros, their scales are set to 1.  Scales go through registers (their rows, K
// / 32 bytes long, have any alignment): thread t fetches those of row t % 256
// of A or B and stores the even blocks' and the odd blocks' in a run each: lane
// half h's scales of the k-steps.
// The stream of K-tiles runs on over the tiles: the last NST K-tiles of a tile
// fetch the first ones of the workgroup's next tile, and the epilogue works
// from registers alone, so that its stores and the next tile's first loads
// overlap.
// What bounds it, by leaving parts out (16384 rows in 32 groups x 4096 x 7168,
// 256 CUs): e2m1 rows 283 us (3.4 PFLOP/s), with every operand read from L2
// again and again 254, without the MFMAs 254, without both 164; the MFMAs alone
// would take 159, at the 6.05 PFLOP/s that random codes sustain, the chip being
// power-limited.  e4m3 rows 411 us (390 on another chip), 383, 330, 214 and, at
// 3.8 PFLOP/s, 253.  So the operands'
// way through L2 and LDS and the MFMAs, each near the half of it, overlap in part,
// and misses in L2 cost the rest.  An L2 prefetch two K-tiles ahead made it 5%
// (weights alone, shared out) to 15% slower: the requests of a CU are scarce.
// For the same reason a round's scales are one load (e4m3 446 -> 421 us against
// a load per K-tile).  64 KB of aligned 128-byte row pieces take 0.53 us from
// L2, of 64-byte pieces or of pieces that straddle lines (K % 256 != 0) 1.0 us:
// four stages of 128 values were 20% slower for e2m1 rows for that reason, three
// of them 5% faster than two for e4m3 rows, of which only the weights take
// 64-byte pieces.
template <bool A4>
__global__ __launch_bounds__(512, 1) void mx4_gemm_tile_kernel(Mx4Args p) {
  constexpr int NST = A4 ? 2 : 3;         // stages
  constexpr int KB = A4 ? 8 : 4;          // blocks of 32 values per K-tile
  constexpr int KSN = KB / 2;             // k-steps per K-tile
  constexpr int NJB = A4 ? 4 : 2;         // DMA pieces (1 KB) of B per wave and K-tile; of A: 4
  constexpr uint32_t kDrop = 0xFFFFFFF0u; // an offset behind every range
  constexpr int ABYTES = 32768;           // A's part of a stage, B's after it
  constexpr int SBYTES = ABYTES + 8192 * NJB;
  // One array per stage, so that the compiler can tell the DMA of one from the
  // reads of another.
  __shared__ __attribute__((aligned(16))) uint8_t st0[SBYTES], st1[SBYTES], st2[NST > 2 ? SBYTES : 16];
  __shared__ __attribute__((aligned(16))) uint8_t sc0[512 * KB], sc1[512 * KB], sc2[NST > 2 ? 512 * KB : 16];
  __shared__ RowScan gs;
  auto stage = [&](auto ic) -> uint8_t* {
    constexpr int i = decltype(ic)::value % NST;
    if constexpr (i == 0) return st0;
    else if constexpr (i == 1) return st1;
    else return st2;
  };
  auto scales = [&](auto ic) -> uint8_t* {
    constexpr int i = decltype(ic)::value % NST;
    if constexpr (i == 0) return sc0;
    else if constexpr (i == 1) return sc1;
    else return sc2;
  };
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  build_row_scan<512, MX4_BM>(gs, p.counts, p.E, p.M_cap, p.offsets_out, p.status_out, blockIdx.x == 0);
  const int NT = (p.N + MX4_BN - 1) / MX4_BN;
  const int nblk = p.K >> 5;                                        // blocks of 32 values
  const int nk = ((nblk + KB - 1) / KB + NST - 1) / NST * NST;      // K-tiles, rounded up by masked ones
  const uint32_t lda = A4 ? (uint32_t)p.K >> 1 : (uint32_t)p.K, ldb = (uint32_t)p.K >> 1;   // bytes per row
  const long long total = (long long)__builtin_amdgcn_readfirstlane(gs.tile_off[p.E]) * NT;
  const int P = gridDim.x;
  // workgroups are dealt to the 8 XCDs in turn: each XCD gets a run of tiles
  const int slot = (P % 8 == 0) ? ((blockIdx.x & 7) * (P >> 3) + (blockIdx.x >> 3)) : blockIdx.x;

  // (carried from tile to tile in vector registers, whatever the compiler may
  // know: scalars again where they are used, see uniform)
  struct Tile { int e, row0, rows, n0; };
  auto uniform = [](const Tile& t) {
    Tile u;
    u.e = __builtin_amdgcn_readfirstlane(t.e);
    u.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    u.rows = __builtin_amdgcn_readfirstlane(t.rows);
    u.n0 = __builtin_amdgcn_readfirstlane(t.n0);
    return u;
  };
  auto decode = [&](long long tile) {
    int lo = 0, hi = p.E;   // the last e with tile_off[e] * NT <= tile
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)gs.tile_off[mid] * NT <= tile) lo = mid; else hi = mid;
    }
    const int t_off = gs.tile_off[lo], MT = gs.tile_off[lo + 1] - t_off;
    const int local = (int)(tile - (long long)t_off * NT);
    // blocks of 4 m-tiles x 8 n-tiles, m fastest: the run of tiles that an
    // XCD works on together shares few panels of either operand
    constexpr int BHT = 4, BWT = 8;
    const int band = local / (BHT * NT);
    const int bh = min(BHT, MT - band * BHT);
    const int l2 = local - band * BHT * NT;
    const int nb = l2 / (bh * BWT);
    const int l3 = l2 - nb * bh * BWT;
    const int mt = band * BHT + l3 % bh, nt = nb * BWT + l3 / bh;
    Tile t;
    t.e = lo;
    t.row0 = gs.row_off[lo] + mt * MX4_BM;
    t.rows = min(MX4_BM, gs.row_off[lo + 1] - t.row0);
    t.n0 = nt * MX4_BN;
    return t;
  };

  // ---- the fetching side: the operands of one tile
  const int srow = tid & 255;
  const bool isA = wave < 4;
  struct Fetch { rsrc_t A, B; const uint8_t* sp; int s_off, s_end; };
  auto fetch_of = [&](const Tile& t, bool any) {
    const int cols = min(MX4_BN, p.N - t.n0);
    const long long brow0 = (long long)t.e * p.N + t.n0;
    Fetch f;
    f.A = make_rsrc(p.A + (long long)t.row0 * lda, any ? (long long)t.rows * lda : 0);
    f.B = make_rsrc(p.B + brow0 * ldb, any ? (long long)cols * ldb : 0);
    // (rows and columns past the end take the last one's scales: what they
    // scale is not stored)
    f.sp = isA ? p.a_scales + (long long)t.row0 * nblk : p.b_scales + brow0 * nblk;
    f.s_off = (isA ? min(srow, t.rows - 1) : min(mx4_col(srow), cols - 1)) * nblk;
    const long long left = (isA ? (long long)p.M_cap - t.row0 : (long long)p.E * p.N - brow0) * nblk;
    f.s_end = (int)min(left, 1LL << 30) - KB * NST;   // the last offset a load may start at
    return f;
  };
  // DMA piece: 1 KB of LDS, 8 rows of 128 bytes or 16 of 64; a lane lands on
  // row l / 8 (l / 4) of it and fetches the logical chunk that its physical one
  // holds.  The address is linear in the piece's row and the lane's: mx4_col(8
  // x + y) = mx4_col(8 x) + mx4_col(y) for y < 8 (and so with 16).  The lane's
  // part is derived anew for each K-tile (opaque zero): registers are what the
  // main loop is short of.
  struct LanePart { uint32_t la, lb; int ca, cb; };
  auto lane_part = [&]() {
    const int l = lane + opaque_zero(), rl = l >> 3;
    LanePart d;
    d.ca = (l & 7) ^ rl;                                  // swz_off, but for the piece's part
    d.cb = A4 ? d.ca : (l & 3) ^ ((l >> 4) & 3);          // mx4_off64
    d.la = (uint32_t)rl * lda;
    d.lb = (uint32_t)mx4_col(A4 ? rl : l >> 2) * ldb;
    return d;
  };
  auto dmaA = [&](const LanePart& d, const Fetch& f, int kt, uint8_t* st, int j) {
    const int piece = wave * 4 + j;
    const int c = d.ca ^ swz_hi(piece & 3);
    const uint32_t off = d.la + (uint32_t)(c * 16) + ((uint32_t)(piece * 8) * lda + (uint32_t)(kt * 128));
    const int left = (nblk - KB * kt) * (A4 ? 1 : 2);     // chunks of the row that are left
    lds_dma16(f.A, st + piece * 1024, c < left ? off : kDrop, 0);
  };
  auto dmaB = [&](const LanePart& d, const Fetch& f, int kt, uint8_t* st, int j) {
    const int piece = wave * NJB + j;
    const int c = A4 ? d.cb ^ swz_hi(piece & 3) : d.cb;
    const int urow = mx4_col(piece * (A4 ? 8 : 16));
    const uint32_t off = d.lb + (uint32_t)(c * 16) + ((uint32_t)urow * ldb + (uint32_t)(kt * (A4 ? 128 : 64)));
    lds_dma16(f.B, st + ABYTES + piece * 1024, c < nblk - KB * kt ? off : kDrop, 0);
  };
  // scales of row srow, those of a round's NST K-tiles with one load: a wave's 64
  // rows are 64 lines of memory however few bytes of each are taken.  The bytes
  // may run over into the next rows, whose are masked; behind the array's last
  // row the load is shifted down.  No branch: with one in the main loop the
  // compiler sinks a k-step's MFMAs below it and spills the fragments.  The
  // bytes are worked on when they are stored, K-tiles after their load.
  constexpr int SW = KB * NST / 4;
  struct Scales { uint32_t w[SW]; int sh; };
  Scales sv;
  auto scale_load = [&](const Fetch& f, int kt) {
    const int want = f.s_off + KB * kt, at = min(want, f.s_end);
    Scales v;
    __builtin_memcpy(v.w, f.sp + at, 4 * SW);
    v.sh = want - at;
    return v;
  };
  // the scales of the load's K-tile j, which is K-tile kt of its row
  auto scale_store = [&](uint8_t* sc, const Scales& v, auto jc, int kt) {
    constexpr int j = decltype(jc)::value;
    // 4 bytes from byte 4 i + sh on (what is behind the load is behind the row)
    auto word = [&](int i) {
      uint32_t lo = v.w[i], hi = i + 1 < SW ? v.w[i + 1] : 0;
#pragma unroll
      for (int o = 1; i + o < SW; ++o) {
        lo = v.sh >> 2 >= o ? v.w[i + o] : lo;
        hi = v.sh >> 2 >= o ? (i + o + 1 < SW ? v.w[i + o + 1] : 0) : hi;
      }
      return __builtin_amdgcn_alignbyte(hi, lo, v.sh & 3);
    };
    const int here = min(max(nblk - KB * kt, 0), KB);   // blocks that the row has; the others: 1 (byte 127)
    auto mask = [&](uint32_t w, int n) {
      const uint32_t m = n >= 4 ? ~0u : (1u << (8 * max(n, 0))) - 1;
      return (w & m) | (0x7F7F7F7Fu & ~m);
    };
    if constexpr (A4) {
      const uint32_t lo4 = mask(word(2 * j), here), hi4 = mask(word(2 * j + 1), here - 4);
      *reinterpret_cast<uint2*>(sc + tid * 8) = make_uint2(__builtin_amdgcn_perm(hi4, lo4, 0x06040200u),
                                                           __builtin_amdgcn_perm(hi4, lo4, 0x07050301u));
    } else {
      const uint32_t w = mask(word(j), here);
      *reinterpret_cast<uint32_t*>(sc + tid * 4) = __builtin_amdgcn_perm(w, w, 0x03010200u);
    }
  };

  long long tile = slot;
  if (tile >= total) return;   // (the whole workgroup)
  Tile cur_ = decode(tile);
  {
    const Fetch f = fetch_of(uniform(cur_), true);
    const LanePart d = lane_part();
    sv = scale_load(f, 0);
    static_for<NST>([&](auto i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) dmaA(d, f, i, stage(i), j);
#pragma unroll
      for (int j = 0; j < NJB; ++j) dmaB(d, f, i, stage(i), j);
    });
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    static_for<NST>([&](auto i) { scale_store(scales(i), sv, i, i); });
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    __syncthreads();
  }

  for (;;) {
    // K-tile 0 of the tile is in stage 0, K-tiles 1 .. NST - 1 are on their way
    // to the other stages; the scales of all of them are stored.  Behind them the
    // last tile's stores may be on their way
    const long long ntile = tile + P;
    const bool more = ntile < total;
    Tile nxt_ = cur_;
    if (more) nxt_ = decode(ntile);
    const Tile cur = uniform(cur_), nxt = uniform(nxt_);

    auto tile_body = [&](auto mic) {
      constexpr int MI = decltype(mic)::value;      // 32-row blocks per wave: 2, or 1 for up to 128 rows
      const int lane_t = lane + opaque_zero();
      const int h = lane_t >> 5;
      const int ra = wm * 32 * MI + (lane_t & 31), rb = wn * 128 + (lane_t & 31);
      using fragA = std::conditional_t<A4, i32x4, i32x8>;
      auto rdA = [&](const uint8_t* st, int ks, int i) -> fragA {
        if constexpr (A4) {
          return *reinterpret_cast<const i32x4*>(st + swz_off(ra + 32 * i, 2 * ks + h));
        } else {   // bytes 16 h .. + 15 of each of the k-step's two blocks
          const i32x4 lo4 = *reinterpret_cast<const i32x4*>(st + swz_off(ra + 32 * i, 4 * ks + h));
          const i32x4 hi4 = *reinterpret_cast<const i32x4*>(st + swz_off(ra + 32 * i, 4 * ks + 2 + h));
          return __builtin_shufflevector(lo4, hi4, 0, 1, 2, 3, 4, 5, 6, 7);
        }
      };
      auto rdB = [&](const uint8_t* st, int ks, int j) {
        const int r = rb + 32 * j, c = 2 * ks + h;
        return *reinterpret_cast<const i32x4*>(st + ABYTES + (A4 ? swz_off(r, c) : mx4_off64(r, c)));
      };
      using sw_t = std::conditional_t<A4, uint32_t, uint16_t>;   // a lane half's scales of a K-tile
      auto rdSA = [&](const uint8_t* sc, int i) { return (int)reinterpret_cast<const sw_t*>(sc)[(ra + 32 * i) * 2 + h]; };
      auto rdSB = [&](const uint8_t* sc, int j) {
        return (int)reinterpret_cast<const sw_t*>(sc)[(256 + rb + 32 * j) * 2 + h];
      };
      f32x16 acc[MI][4];
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
      fragA aF[2][MI];
      i32x4 bF[4];
      int sA[MI], sB[4], nA[MI], nB[4];
      auto operandA = [](const fragA& v) {
        if constexpr (A4) return mx4_frag(v);
        else return v;
      };
      // one k-step (KS) of the K-tile in stage S, B block j outer: fragment j is
      // dead after its MI MFMAs and is read again for the next k-step at once;
      // the next A fragments go into the other buffer.  The last k-step reads the
      // next stage's fragments and scales, and issues the DMA of K-tile dkt of
      // ff into its own stage.
      auto kstep = [&](auto ksc, auto sc_, const Fetch& ff, int dkt) {
        constexpr int KS = decltype(ksc)::value, S = decltype(sc_)::value;
        constexpr bool LAST = KS == KSN - 1;
        constexpr int NK = (KS + 1) % KSN;
        using NS = std::integral_constant<int, (S + (LAST ? 1 : 0)) % NST>;
        LanePart d;
        if constexpr (LAST) d = lane_part();
        static_for<4>([&](auto jc) {
          constexpr int j = decltype(jc)::value;
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (j < MI) aF[(KS + 1) & 1][j] = rdA(stage(NS{}), NK, j);
          if constexpr (LAST) {
            if constexpr (j < MI) nA[j] = rdSA(scales(NS{}), j);
            nB[j] = rdSB(scales(NS{}), j);
            if constexpr (A4) {
              if constexpr (j < 2) {
                dmaA(d, ff, dkt, stage(sc_), 2 * j);
                dmaA(d, ff, dkt, stage(sc_), 2 * j + 1);
              } else {
                dmaB(d, ff, dkt, stage(sc_), 2 * j - 4);
                dmaB(d, ff, dkt, stage(sc_), 2 * j - 3);
              }
            } else {
              dmaA(d, ff, dkt, stage(sc_), j);
              if constexpr (j >= 2) dmaB(d, ff, dkt, stage(sc_), j - 2);
            }
          }
          static_for<MI>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                mx4_frag(bF[j]), operandA(aF[KS & 1][i]), acc[i][j], 4, A4 ? 4 : 0, KS, sB[j], KS, sA[i]);
          });
          bF[j] = rdB(stage(NS{}), NK, j);
        });
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (LAST) {
#pragma unroll
          for (int i = 0; i < MI; ++i) sA[i] = nA[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) sB[j] = nB[j];
        }
      };
      // K-tiles kt .. kt + NST - 1; fetches K-tiles fkt .. of ff.  Before the
      // last k-step of each: K-tile kt + s + 1 has landed (the DMA of the NST -
      // 2 after it may be on its way; with their scales' loads that is less than
      // what is, and waits for the oldest of them too), its scales are stored,
      // and every wave's reads of stage s are done.  FIRST: the tile's first
      // round, whose K-tiles' scales are stored.  The last tile's stores came
      // after its K-tiles' DMA and are waited for with them: their number is the
      // compiler's choice (it merges and drops stores), so no count may rest on it.
      auto round = [&](auto first, int kt, const Fetch& ff, int fkt) {
        constexpr bool FIRST = decltype(first)::value;
        static_for<NST>([&](auto sc_) {
          constexpr int S = decltype(sc_)::value, NX = (S + 1) % NST;
          static_for<KSN - 1>([&](auto ks) { kstep(ks, sc_, ff, 0); });
          constexpr bool BEFORE = FIRST && S < NST - 1;
          constexpr int VM = (NST - 2) * (4 + NJB);
          __builtin_amdgcn_s_waitcnt(0x0F70 | (VM & 15) | ((VM >> 4) << 14));   // vmcnt(VM)
          if constexpr (!BEFORE)
            scale_store(scales(std::integral_constant<int, NX>{}), sv, std::integral_constant<int, NX>{},
                        S == NST - 1 ? fkt : kt + S + 1);
          // (the bare barrier: __syncthreads would wait for all loads)
          asm volatile("" ::: "memory");
          __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (S == NST - 2) sv = scale_load(ff, fkt);   // (the last of the round before is stored)
          kstep(std::integral_constant<int, KSN - 1>{}, sc_, ff, fkt + S);
        });
      };
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < MI; ++i) { aF[0][i] = rdA(st0, 0, i); sA[i] = rdSA(sc0, i); }
#pragma unroll
      for (int j = 0; j < 4; ++j) { bF[j] = rdB(st0, 0, j); sB[j] = rdSB(sc0, j); }
      // the operands that the round from K-tile kt on fetches: those behind it,
      // or at the end the next tile's (after the last tile its loads read nothing)
      auto fetch_at = [&](int kt) {
        const bool end = kt + NST >= nk;
        Tile t;
        t.e = end ? nxt.e : cur.e;
        t.row0 = end ? nxt.row0 : cur.row0;
        t.rows = end ? nxt.rows : cur.rows;
        t.n0 = end ? nxt.n0 : cur.n0;
        return fetch_of(t, !end || more);
      };
      round(std::true_type{}, 0, fetch_at(0), NST < nk ? NST : 0);
      for (int kt = NST; kt < nk; kt += NST) round(std::false_type{}, kt, fetch_at(kt), kt + NST < nk ? kt + NST : 0);
      // the sums are needed here: without this the compiler sinks the last
      // MFMAs into the epilogue's branches, with their fragments in scratch
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(acc[i][j]));
      // lane (r, h) holds, of row r, columns 8 h .. + 7 of the first and of the
      // second 16 of each 32; the swap gives lanes r and r + 16 the two halves
      // of one row, so that a store covers 64 bytes of each of 16 rows
      const int z = opaque_zero(), le = lane + z;
      const int er = le & 15, eo = 16 * ((le >> 4) & 1) + 8 * (le >> 5);
      const rsrc_t C = make_rsrc(p.C + (long long)cur.row0 * p.N + cur.n0, (long long)cur.rows * p.N * 2 - cur.n0 * 2LL);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const uint32_t row = (uint32_t)(wm * 32 * MI + 32 * i + er) * ((uint32_t)p.N * 2) + 2 * eo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = wn * 128 + 32 * j;
          uint32_t w[8];
#pragma unroll
          for (int d = 0; d < 8; ++d) w[d] = pack_bf16x2(acc[i][j][2 * d], acc[i][j][2 * d + 1]);
#pragma unroll
          for (int d = 0; d < 4; ++d) swap16(w[d], w[4 + d]);
          const uint32_t off = n < p.N - cur.n0 ? row + 2 * n : kDrop;
          const uint32_t off16 = n < p.N - cur.n0 ? off + 16 * ((uint32_t)p.N * 2) : kDrop;
          __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[0], w[1], w[2], w[3]}, C, off, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[4], w[5], w[6], w[7]}, C, off16, 0, 0);
        }
      }
      static_for<NST - 1>([&](auto i) {
        constexpr std::integral_constant<int, decltype(i)::value + 1> s{};
        scale_store(scales(s), sv, s, s);
      });
    };
    if (cur.rows > 128) tile_body(std::integral_constant<int, 2>{});
    else tile_body(std::integral_constant<int, 1>{});
    if (!more) break;
    cur_ = nxt_;
    tile = ntile;
  }
}

}  // namespace moe
