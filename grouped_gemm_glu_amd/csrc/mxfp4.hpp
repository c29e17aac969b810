// MXFP4: OCP e2m1 codes in blocks of 32 values with one E8M0 scale, their
// quantisation and their grouped product on the block-scaled MFMA.
#pragma once

#include "device_common.hpp"
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

// Row-wise quantisation of a bf16 [R][C] matrix: 4 lanes per 32-value block,
// 16 bytes read and 4 bytes of codes written per lane.  A block holding a NaN
// or an infinity gets the NaN scale 0xFF and zero codes (e2m1 has no NaN).
__global__ __launch_bounds__(256) void mx4_rows_kernel(const uint16_t* __restrict__ v, int R, int C,
                                                       const int* __restrict__ counts, int E,
                                                       uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  __shared__ GroupScan gs;
  int rows = R;
  if (counts) {
    build_group_scan<256>(gs, counts, E, R, 1, 0, nullptr, nullptr, false);
    rows = gs.row_off[E];
  }
  const long long total = (long long)rows * (C >> 3);   // a multiple of 4
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const uint4 u = reinterpret_cast<const uint4*>(v)[i];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float x[8];
    float amax = 0.0f;
    int nan = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      amax = fmaxf(amax, fabsf(x[j]));
      nan |= x[j] != x[j];
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      amax = fmaxf(amax, __shfl_xor(amax, d, 64));
      nan |= __shfl_xor(nan, d, 64);
    }
    const int X = nan ? 128 : mx4_scale_exponent(amax);
    reinterpret_cast<uint32_t*>(q)[i] = X == 128 ? 0u : e2m1x8(x, pow2f(X));
    if ((i & 3) == 0) s[i >> 2] = e8m0_byte(X);
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

// Grouped product straight from memory: one workgroup per (16 MB rows of a
// group, 16 columns), its 4 waves sharing K in steps of 128 values; the
// partial sums are added through LDS in wave order.  Lane (r, q) = (l % 16,
// l / 16) of v_mfma_scale_f32_16x16x128_f8f6f4 holds, of an e2m1 operand, row
// r's block q (16 bytes) with its scale; of an e4m3 operand, bytes 16 q .. + 15
// of the step's first 64 values and of its second 64, and the scale of block q.
// The result's lane holds columns 4 q .. + 3 of row r.
template <bool A4, int MB>
__global__ __launch_bounds__(256) void mx4_gemm_small_kernel(Mx4Args p) {
  __shared__ GroupScan gs;
  __shared__ f32x4 red[3][MB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  build_group_scan<256>(gs, p.counts, p.E, p.M_cap, 16 * MB, 0, p.offsets_out, p.status_out, blockIdx.x == 0);
  const int ncb = p.N >> 4, nblk = p.K >> 5;
  const long long items = (long long)gs.tile_off[p.E] * ncb;
  const long long ldb = p.K >> 1, lda = A4 ? p.K >> 1 : p.K;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int tile = (int)(it / ncb), n0 = (int)(it - (long long)tile * ncb) * 16;
    int lo = 0, hi = p.E;   // the last e with tile_off[e] <= tile
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (gs.tile_off[mid] <= tile) lo = mid; else hi = mid;
    }
    const int row0 = gs.row_off[lo] + (tile - gs.tile_off[lo]) * 16 * MB;
    const int rows = min(16 * MB, gs.row_off[lo + 1] - row0);
    const long long brow = (long long)lo * p.N + n0 + r;
    f32x4 acc[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int ks = wave * 4; ks < nblk; ks += 16) {   // first block of the step
      const int b = ks + q;
      i32x8 bv = {0, 0, 0, 0, 0, 0, 0, 0};
      int sb = 127;
      if (b < nblk) {
        const int4 u = *reinterpret_cast<const int4*>(p.B + brow * ldb + b * 16);
        bv[0] = u.x; bv[1] = u.y; bv[2] = u.z; bv[3] = u.w;
        sb = p.b_scales[brow * nblk + b];
      }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const long long arow = row0 + m * 16 + r;
        const bool in = m * 16 + r < rows;
        i32x8 av = {0, 0, 0, 0, 0, 0, 0, 0};
        int sa = 127;
        if (in && b < nblk) sa = p.a_scales[arow * nblk + b];
        if constexpr (A4) {
          if (in && b < nblk) {
            const int4 u = *reinterpret_cast<const int4*>(p.A + arow * lda + b * 16);
            av[0] = u.x; av[1] = u.y; av[2] = u.z; av[3] = u.w;
          }
        } else {
          const int b0 = ks + (q >> 1), b1 = b0 + 2;   // the blocks of this lane's two 16-byte pieces
          const uint8_t* ap = p.A + arow * lda + (long long)b0 * 32 + (q & 1) * 16;
          if (in && b0 < nblk) {
            const int4 u = *reinterpret_cast<const int4*>(ap);
            av[0] = u.x; av[1] = u.y; av[2] = u.z; av[3] = u.w;
          }
          if (in && b1 < nblk) {
            const int4 u = *reinterpret_cast<const int4*>(ap + 64);
            av[4] = u.x; av[5] = u.y; av[6] = u.z; av[7] = u.w;
          }
        }
        acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc[m], 4, A4 ? 4 : 0, 0, sb, 0, sa);
      }
    }
    __syncthreads();   // the previous item's sums are read
    if (wave > 0)
#pragma unroll
      for (int m = 0; m < MB; ++m) red[wave - 1][m][lane] = acc[m];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if (m * 16 + r >= rows) continue;
        const f32x4 v = acc[m] + red[0][m][lane] + red[1][m][lane] + red[2][m][lane];
        *reinterpret_cast<uint2*>(p.C + (long long)(row0 + m * 16 + r) * p.N + n0 + 4 * q) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    }
  }
}

}  // namespace moe
