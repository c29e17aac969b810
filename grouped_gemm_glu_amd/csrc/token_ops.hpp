// Kernels over tokens around the expert GEMMs: the router (scores, balance
// bias, expert groups, top-k, weights) and its gradient, the combine of a
// token's expert rows and its gradients, and the residual addition +
// root-mean-square norm with an MXFP8 copy and its gradients.  All but the
// router read and write each byte once and are bound by memory; the router is
// bound by the instructions of its selection.
#pragma once

#include "device_common.hpp"
#include "operator_args.hpp"

namespace moe {

// ---------------------------------------------------------------- router
// A value's rank as an unsigned integer: larger means earlier in the order.
// NaN ranks below every number (1); 0 is kept for what is out of the choice.
// The two zeros are the same value (v + 0.0 turns -0.0 into +0.0).
__device__ __forceinline__ unsigned long long rank_key(double v) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, v + 0.0);
  const unsigned long long s = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return v != v ? 1ull : s;
}

// Another lane's value by data-parallel primitives (a few cycles each, where a
// shuffle through LDS takes over a hundred); rows not in ROWS get `other`.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t v, uint32_t other = 0) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)other, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float v, float other = 0.0f) {
  return __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(v), __float_as_uint(other)));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp(double v) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
  const unsigned long long o = (unsigned long long)dpp<CTRL, ROWS>((uint32_t)(b >> 32)) << 32 |
                               dpp<CTRL, ROWS>((uint32_t)b);
  return __builtin_bit_cast(double, o);
}
__device__ __forceinline__ uint32_t lane63(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }

// Over a whole wave (all lanes active): rotations within the rows of 16 lanes,
// then lane 15 of rows 0 and 2 to rows 1 and 3, lane 31 to rows 2 and 3.
template <class V>
__device__ __forceinline__ V wave_sum_to_lane63(V v) {
  v += dpp<0x128>(v);
  v += dpp<0x124>(v);
  v += dpp<0x122>(v);
  v += dpp<0x121>(v);
  v += dpp<0x142, 0xA>(v);
  v += dpp<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(lane63(__float_as_uint(wave_sum_to_lane63(v))));
}
__device__ __forceinline__ double wave_sum(double v) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, wave_sum_to_lane63(v));
  return __builtin_bit_cast(double, (unsigned long long)lane63((uint32_t)(b >> 32)) << 32 | lane63((uint32_t)b));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp<0x128>(v));
  v = max(v, dpp<0x124>(v));
  v = max(v, dpp<0x122>(v));
  v = max(v, dpp<0x121>(v));
  v = max(v, dpp<0x142, 0xA>(v));
  v = max(v, dpp<0x143, 0xC>(v));
  return lane63(v);
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0x128>(v));
  v = fmaxf(v, dpp<0x124>(v));
  v = fmaxf(v, dpp<0x122>(v));
  v = fmaxf(v, dpp<0x121>(v));
  v = fmaxf(v, dpp<0x142, 0xA>(v, -INFINITY));
  v = fmaxf(v, dpp<0x143, 0xC>(v, -INFINITY));
  return __uint_as_float(lane63(__float_as_uint(v)));
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, long long i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// One token by a whole wave, experts lane, lane + 64, ...: k rounds of a
// wave-wide maximum.  Scores and choice values are kept in 64 bits, so that
// the choice is the one that the formulas make: in 32 bits the scores of
// neighbouring logits round to one value and the order is lost.  tmp: 64 VPL
// doubles of LDS that are this wave's alone.
template <int VPL, bool BF16>
__device__ void router_token_exact(const RouterArgs& p, long long tok, double* tmp, int* __restrict__ ids,
                                   float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  float x[VPL];
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < p.E ? load_logit<BF16>(p.logits, tok * p.E + e) : -INFINITY;
    m = fmaxf(m, x[i]);
    nan = nan || x[i] != x[i];
  }
  // softmax: the maximum and the sum over the row (a NaN logit makes the sum
  // NaN; a row of -inf alone has no softmax, its scores are 0)
  m = wave_max(m);
  const bool empty = m == -INFINITY && !__any(nan);
  double sum = 1.0;
  if (!p.sigmoid) {
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i < p.E) sum += exp((double)x[i] - (double)m);
    sum = wave_sum(sum);
  }
  auto score = [&](float v) -> double {
    if (p.sigmoid) return 1.0 / (1.0 + exp(-(double)v));
    return empty ? 0.0 : exp((double)v - (double)m) / sum;
  };
  // the choice value: score + bias, or without a bias the logit itself (the
  // same order without the scores' rounding)
  const bool by_score = p.bias != nullptr || (p.n_groups > 1 && p.top2);
  double c[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    c[i] = -INFINITY;
    if (e < p.E) c[i] = by_score ? score(x[i]) + (p.bias ? (double)p.bias[e] : 0.0) : (double)x[i];
  }
  unsigned long long open = ~0ull;   // bit g: group g takes part
  if (p.n_groups > 1) {
    const int gsz = p.E / p.n_groups;
#pragma unroll
    for (int i = 0; i < VPL; ++i) tmp[lane + 64 * i] = c[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    unsigned long long key = 0;
    if (lane < p.n_groups) {
      double b0 = -INFINITY, b1 = -INFINITY;
      bool num = false, num2 = false;   // a first and a second number in the group
#pragma unroll 8
      for (int i = 0; i < gsz; ++i) {
        double v = tmp[lane * gsz + i];
        const bool is = v == v;
        v = is ? v : -INFINITY;
        num2 = num2 || (num && is);
        num = num || is;
        b1 = fmax(b1, fmin(b0, v));
        b0 = fmax(b0, v);
      }
      if (p.top2) key = num2 ? rank_key(b0 + b1) : 1ull;
      else key = num ? rank_key(b0) : 1ull;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // (tmp may be the next token's)
    int before = 0;
    for (int g = 0; g < p.n_groups; ++g) {
      const unsigned long long o = __shfl(key, g, 64);
      before += o > key || (o == key && g < lane);
    }
    open = __ballot(lane < p.n_groups && before < p.topk_groups);
    if (!p.bias && p.top2) {   // without a bias the experts' order is the logits'
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = (double)x[i];
    }
  }
  unsigned long long key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    const bool in = e < p.E && (p.n_groups == 1 || ((open >> (e / (p.E / p.n_groups))) & 1ull));
    key[i] = in ? rank_key(c[i]) : 0ull;
  }
  int my_id = 0;
  for (int j = 0; j < p.k; ++j) {
    unsigned long long b = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) b = key[i] > b ? key[i] : b;
    const uint32_t hi = wave_max((uint32_t)(b >> 32));
    const uint32_t lo = wave_max((uint32_t)(b >> 32) == hi ? (uint32_t)b : 0u);
    b = (unsigned long long)hi << 32 | lo;
    uint32_t at = 0;   // ~expert: the lowest of equals
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i) at = key[i] == b ? ~(uint32_t)(lane + 64 * i) : at;
    const int e = (int)~wave_max(at);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i == e) key[i] = 0;
    if (lane == j) my_id = e;
  }
  const float my_x = lane < p.k ? load_logit<BF16>(p.logits, tok * p.E + my_id) : 0.0f;
  const double s = lane < p.k ? score(my_x) : 0.0;
  const double total = p.renorm ? wave_sum(s) : 1.0;
  if (lane < p.k) {
    ids[tok * p.k + lane] = my_id;
    weights[tok * p.k + lane] = total == 0.0 ? 0.0f : (float)((double)p.scale * s / total);
  }
}

// Every token by the exact routine: for what the fast kernel does not take
// (E % 4 != 0, groups of other sizes than 4, 8, 16, ... experts).
template <int VPL, bool BF16>
__global__ __launch_bounds__(256) void router_exact_kernel(RouterArgs p, int* __restrict__ ids,
                                                           float* __restrict__ weights) {
  __shared__ double tmp[4][64 * VPL];
  const int wave = threadIdx.x >> 6;
  const long long tok = (long long)blockIdx.x * 4 + wave;
  if (tok < p.T) router_token_exact<VPL, BF16>(p, tok, tmp[wave], ids, weights);
}

// Maximum (minimum) over the L lanes of a token, which all get it: rotations
// within each row of 16 lanes, then across the rows.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (L == 64) return wave_max(v);
  v = max(v, dpp<0x128>(v));
  v = max(v, dpp<0x124>(v));
  v = max(v, dpp<0x122>(v));
  v = max(v, dpp<0x121>(v));
  if constexpr (L == 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
  return v;
}
template <int L>
__device__ __forceinline__ int lanes_min(int v) { return (int)~lanes_max<L>(~(uint32_t)v); }
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  static_assert(L >= 16, "rows of 16 lanes");
  if constexpr (L == 64) return wave_sum(v);
  v += dpp<0x128>(v);
  v += dpp<0x124>(v);
  v += dpp<0x122>(v);
  v += dpp<0x121>(v);
  if constexpr (L == 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// As rank_key, of 32-bit values.
__device__ __forceinline__ uint32_t rank_key32(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return v != v ? 1u : ((b >> 31) ? ~b : (b | 0x80000000u));
}
__device__ __forceinline__ float of_rank_key32(uint32_t k) {
  return k <= 1u ? __builtin_nanf("") : __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

// 64 / L tokens per wave, L lanes each; lane l holds experts 4 (l + L i) .. + 3, i
// < NI.  The choice is made on 32-bit values: without a bias (and without sums
// of scores for groups) these are the logits, and exact.  Where scores decide,
// their 32-bit forms are off by at most 2^-21.4 max(1, |c|) for a sigmoid (its
// exponential by (|x| + 2) 2^-24 of itself, s (1 - s) |x| <= 0.23, a quotient and
// two sums), 2^-19.5 for a softmax (a sum of E terms, in 20 roundings); a token
// with two neighbours among its k + 1 best closer than twice that (and a
// little), or a kept and another group whose values are not further apart than
// their errors (twice that each, and the sum's rounding), is done again in 64 bits
// by the whole wave.
// Bound by instructions and their latency: a round of the choice is about 80 for
// 64 / L tokens.  256 experts in 8 groups, k = 8, sigmoid and bias: one token 4.9
// us (a launch that does nothing takes 3.6), 16384 tokens 20 us, of which the
// few tokens of 64 bits, whose waves end last, are about 5; 65536 tokens 49 us.
// Without a bias 16384 tokens take 13.5 us, without groups too 9.5, and no token
// of the latter needs 64 bits.  Equal choice values among a token's best are not
// told apart in 32 bits either: a bias of zeros on bf16 logits, which has many, takes
// 44 us.  A token per wave in 64 bits throughout took 55 us, and one token 11.
template <int L, int NI, bool BF16>
__global__ __launch_bounds__(256) void router_kernel(RouterArgs p, int* __restrict__ ids,
                                                     float* __restrict__ weights) {
  constexpr int VPL = (L * NI * 4 + 63) / 64;   // experts per lane of the exact routine
  __shared__ double tmp[4][64 * VPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & (L - 1);
  const long long tok0 = ((long long)blockIdx.x * 4 + wave) * (64 / L);
  const long long tok = tok0 + lane / L;
  const bool tv = tok < p.T;
  const bool by_score = p.bias != nullptr || (p.n_groups > 1 && p.top2);
  float x[NI][4], c[NI][4];   // (c: the bias first)
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = 4 * (l + L * i);
    c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.0f;
    if (p.bias && e < p.E) __builtin_memcpy(c[i], p.bias + e, 16);
    if (tv && e < p.E) {   // (E % 4 == 0: whole quads)
      if constexpr (BF16) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.logits) + tok * p.E + e);
        x[i][0] = __uint_as_float(u.x << 16);
        x[i][1] = __uint_as_float(u.x & 0xFFFF0000u);
        x[i][2] = __uint_as_float(u.y << 16);
        x[i][3] = __uint_as_float(u.y & 0xFFFF0000u);
      } else {
        const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + tok * p.E + e);
        x[i][0] = u.x;
        x[i][1] = u.y;
        x[i][2] = u.z;
        x[i][3] = u.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) x[i][q] = -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      m = fmaxf(m, x[i][q]);
      nan = nan || x[i][q] != x[i][q];
    }
  // softmax: maximum and, where the scores themselves count, the row's sum
  float inv = 1.0f;
  bool empty = false;
  if (!p.sigmoid) {
    m = of_rank_key32(lanes_max<L>(rank_key32(m)));
    const bool any_nan = lanes_max<L>(nan ? 1u : 0u) != 0u;
    empty = m == -INFINITY && !any_nan;
    float sum = any_nan ? __builtin_nanf("") : 1.0f;
    if (by_score || !p.renorm) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (4 * (l + L * i) < p.E) sum += __expf(x[i][q] - m);
      sum = lanes_sum<L>(sum);
    }
    inv = 1.0f / sum;
  }
  bool redo = false;
  // the relative width within which two 32-bit choice values say nothing, and the
  // relative error of a group's sum of two of them (and a little)
  const float tol = p.sigmoid ? 0x1p-20f : 0x1p-18f;
  auto close = [=](float hi, float lo) {   // (true for NaN)
    return !(hi - lo > tol * fmaxf(1.0f, fmaxf(fabsf(hi), fabsf(lo))));
  };
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) c[i][q] = f(x[i][q], c[i][q]);
  };
  if (!by_score) each([](float v, float) { return v; });
  else if (p.sigmoid) each([](float v, float b) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)) + b; });
  else if (!empty) each([=](float v, float b) { return fmaf(__expf(v - m), inv, b); });
  uint32_t open = (1u << NI) - 1;   // bit i: this lane's quad i takes part
  if (p.n_groups > 1) {
    // a group is W = size / 4 neighbouring lanes' quads i (W a power of two up to
    // L): the two best values of the quad, then of the W lanes
    const int W = p.E / p.n_groups / 4, sh = __builtin_ctz(W);
    float v0[NI], v1[NI];
    uint32_t key[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float b0 = fmaxf(c[i][0], c[i][1]), b1 = fminf(c[i][0], c[i][1]);
      const float d0 = fmaxf(c[i][2], c[i][3]), d1 = fminf(c[i][2], c[i][3]);
      b1 = fmaxf(fminf(b0, d0), fmaxf(b1, d1));
      b0 = fmaxf(b0, d0);
      v0[i] = b0;
      v1[i] = b1;
    }
    auto merge = [&](auto other) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float o0 = other(v0[i]), o1 = other(v1[i]);
        v1[i] = fmaxf(fminf(v0[i], o0), fmaxf(v1[i], o1));
        v0[i] = fmaxf(v0[i], o0);
      }
    };
    // lane ^ 1, ^ 2 by quad permutes; then, the quads being alike, the mirrors
    // of 8 and of 16 lanes reach the other quad, the other half row
    if (W > 1) merge([](float v) { return dpp<0xB1>(v); });
    if (W > 2) merge([](float v) { return dpp<0x4E>(v); });
    if (W > 4) merge([](float v) { return dpp<0x141>(v); });
    if (W > 8) merge([](float v) { return dpp<0x140>(v); });
    if (W > 16) merge([](float v) { return __shfl_xor(v, 16, 64); });
    if (W > 32) merge([](float v) { return __shfl_xor(v, 32, 64); });
    // (fmax and fmin drop a NaN, of a logit or of the bias, and the number beside it
    // counts twice: such tokens are done again below)
    bool no_number = false;
    each([&](float, float v) {
      no_number = no_number || v != v;
      return v;
    });
#pragma unroll
    for (int i = 0; i < NI; ++i)
      key[i] = 4 * (l + L * i) < p.E ? rank_key32(p.top2 ? v0[i] + v1[i] : v0[i]) : 0u;
    redo = lanes_max<L>(no_number ? 1u : 0u) != 0u;
    // the kept groups, best first, ties to the lower id
    open = 0;
    for (int g = 0; g < p.topk_groups; ++g) {
      uint32_t b = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) b = max(b, key[i]);
      b = lanes_max<L>(b);
      int at = 0x7FFFFFFF;   // group id
#pragma unroll
      for (int i = NI - 1; i >= 0; --i)
        if (key[i] == b) at = (l + L * i) >> sh;
      at = lanes_min<L>(at);
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if ((l + L * i) >> sh == at) {
          key[i] = 0;
          open |= 1u << i;
        }
    }
    // 32 bits decide if every kept group's value less its error is above every
    // other's with its error, which goes by the two values' own sizes: their sum
    // may cancel.  (A value that is infinite is so in 64 bits too.)
    if (by_score && p.topk_groups < p.n_groups) {
      uint32_t kept = 0, left = 0;   // of -(value - error), of value + error
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (4 * (l + L * i) >= p.E) continue;
        const float v = p.top2 ? v0[i] + v1[i] : v0[i];
        const float err = fabsf(v) < INFINITY ? tol * fmaxf(1.0f, p.top2 ? fmaxf(fabsf(v0[i]), fabsf(v1[i])) : fabsf(v)) : 0.0f;
        if ((open >> i) & 1u) kept = max(kept, rank_key32(err - v));
        else left = max(left, rank_key32(v + err));
      }
      kept = lanes_max<L>(kept);
      left = lanes_max<L>(left);
      redo = redo || !(-of_rank_key32(kept) > of_rank_key32(left));
    }
    if (!p.bias && p.top2) {   // without a bias the experts' order is the logits'
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) c[i][q] = x[i][q];
    }
  }
  const bool check = p.bias != nullptr;   // the choice among experts is by scores
  uint32_t key[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      key[i][q] = ((open >> i) & 1u) && 4 * (l + L * i) < p.E ? rank_key32(c[i][q]) : 0u;
  int my_id = 0;
  float last = 0.0f;
  for (int j = 0; j < p.k + (check ? 1 : 0); ++j) {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) b = max(max(b, max(key[i][0], key[i][1])), max(key[i][2], key[i][3]));
    b = lanes_max<L>(b);
    if (check) {
      const float v = of_rank_key32(b);
      if (j > 0 && b != 0u && close(last, v)) redo = true;
      last = v;
      if (j == p.k) break;
    }
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = NI - 1; i >= 0; --i)
#pragma unroll
      for (int q = 3; q >= 0; --q) at = key[i][q] == b ? 4 * (l + L * i) + q : at;
    at = lanes_min<L>(at);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) key[i][q] = 4 * (l + L * i) + q == at ? 0u : key[i][q];
    if (l == j) my_id = at;
  }
  const bool sel = tv && l < p.k;
  float s = 0.0f;
  // a score, also times the scale, near or below what fp32 holds: its ratio to the
  // others may still count
  bool tiny = false;
  if (sel) {
    const float v = load_logit<BF16>(p.logits, tok * p.E + my_id);
    s = p.sigmoid ? 1.0f / (1.0f + expf(-v)) : (empty ? 0.0f : expf(v - m) * inv);
    tiny = s * fminf(fabsf(p.scale), 1.0f) < 1e-30f && v != -INFINITY && !empty && p.scale != 0.0f;
  }
  redo = redo || lanes_max<L>(tiny ? 1u : 0u) != 0u;
  const float total = p.renorm ? lanes_sum<L>(s) : 1.0f;
  if (sel && !redo) {
    ids[tok * p.k + l] = my_id;
    weights[tok * p.k + l] = total == 0.0f ? 0.0f : p.scale * s / total;
  }
  unsigned long long again = __ballot(tv && redo && l == 0);
  while (again) {
    const int at = __builtin_ctzll(again);
    again &= again - 1;
    router_token_exact<VPL, BF16>(p, tok0 + at / L, tmp[wave], ids, weights);
  }
}

// d(logits) from d(weights) and the ids that were chosen.  With s the scores, w =
// s / S (S = sum of the chosen ones, or 1 without renormalisation), dw the
// weights' gradients and m = sum_i dw_i w_i (0 without renormalisation), the
// chosen experts' part is d_j = scale w_j (dw_j - m), and
//   sigmoid: dx = d_j (1 - s_j) at the chosen experts, 0 elsewhere
//   softmax: dx_e = d_e [e chosen] - s_e sum_i d_i; renormalised softmax is the
//   softmax over the chosen logits, so only those count, and sum_i d_i = 0.
// 1 / S stands only in w: dw / S could pass fp32's range where dx does not.  A
// token with a chosen sigmoid score near or below what fp32 holds has its
// weights formed in 64 bits, as the forward pass does.
// An id outside [0, E) takes no part; an id that stands twice counts twice.
template <int VPL, bool BF16>
__global__ __launch_bounds__(256) void router_bwd_kernel(RouterArgs p, const int* __restrict__ ids,
                                                         const float* __restrict__ dw,
                                                         void* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long tok = (long long)blockIdx.x * 4 + wave;
  if (tok >= p.T) return;   // (no barrier below)
  int id = -1;
  float xs = 0.0f, g = 0.0f;
  if (lane < p.k) {
    id = ids[tok * p.k + lane];
    g = dw[tok * p.k + lane];
    if (id < 0 || id >= p.E) id = -1;
    else xs = load_logit<BF16>(p.logits, tok * p.E + id);
  }
  const bool in = id >= 0;
  float x[VPL];
  float m = -INFINITY, sum = 1.0f;
  bool nan = in && xs != xs;
  const bool full = !p.sigmoid && !p.renorm;   // softmax over the whole row
  if (full) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 64 * i;
      x[i] = e < p.E ? load_logit<BF16>(p.logits, tok * p.E + e) : -INFINITY;
      m = fmaxf(m, x[i]);
      nan = nan || x[i] != x[i];
    }
    m = wave_max(m);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i < p.E) sum += expf(x[i] - m);
    sum = wave_sum(sum);
  } else if (!p.sigmoid) {
    m = wave_max(in ? xs : -INFINITY);
  }
  // A renormalised softmax whose choice is not by logits alone may have chosen
  // experts that are so far below the row's largest logit that their scores are 0
  // in 64 bits, and the weights with them: those rows are looked through.
  bool under = false;
  if (!p.sigmoid && p.renorm && (p.bias || (p.n_groups > 1 && p.top2))) {
    float top = -INFINITY;
    for (int e = lane; e < p.E; e += 64) top = fmaxf(top, load_logit<BF16>(p.logits, tok * p.E + e));
    top = wave_max(top);
    if (m > -INFINITY && m - top < -700.0f) {
      double all = 0.0;
      for (int e = lane; e < p.E; e += 64) all += exp((double)load_logit<BF16>(p.logits, tok * p.E + e) - (double)top);
      all = wave_sum(all);
      under = exp((double)m - (double)top) / all == 0.0;
    }
  }
  float s = 0.0f;
  if (in) s = p.sigmoid ? 1.0f / (1.0f + expf(-xs)) : expf(xs - m) / sum;
  const bool empty = !p.sigmoid && m == -INFINITY && !__any(nan);   // no softmax: constant weights
  if (empty) s = 0.0f;
  float w;
  bool none = empty || under;   // the weights are 0
  if (p.sigmoid && __any(in && s < 1e-30f && xs != -INFINITY)) {
    const double sd = in ? 1.0 / (1.0 + exp(-(double)xs)) : 0.0;
    const double S = p.renorm ? wave_sum(sd) : 1.0;
    none = S == 0.0;
    w = (float)(sd / S);
  } else {
    const float S = p.renorm ? wave_sum(s) : 1.0f;
    none = none || S == 0.0f;
    w = s / S;
  }
  const float mean = p.renorm ? wave_sum(in ? g * w : 0.0f) : 0.0f;
  float d = 0.0f, dot = 0.0f;
  if (in && !none) {
    d = p.scale * w * (g - mean);
    if (p.sigmoid) d *= 1.0f / (1.0f + expf(xs));
  }
  if (full) dot = wave_sum(d);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    float v = full && !empty && e < p.E ? -(expf(x[i] - m) / sum) * dot : 0.0f;
    for (int j = 0; j < p.k; ++j) {
      const int ej = __builtin_amdgcn_readlane(id, j);
      const float dj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(d), j));
      v += ej == e ? dj : 0.0f;
    }
    if (e < p.E) {
      if constexpr (BF16) static_cast<uint16_t*>(dlogits)[tok * p.E + e] = f32_to_bf16(v);
      else static_cast<float*>(dlogits)[tok * p.E + e] = v;
    }
  }
}

// ---------------------------------------------------------------- combine
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// out[t] = residual[t] + sum_j w[t][j] y[dst[t][j]], the terms added in slot
// order in fp32 and rounded once.  One thread per 8 columns of a token, four of
// its rows in flight together.  out may be the residual itself: the thread that
// writes 8 columns has read them.  Bound by memory: 16384 tokens, k = 8, H = 7168,
// 423 us, 5.0 TB/s, as fast as the rows can be read in order (413).
constexpr int kCombineRows = 4;
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ y, int M_cap, int H,
                                                      const int* __restrict__ dst,
                                                      const float* __restrict__ weights, int T, int k,
                                                      const uint16_t* residual, uint16_t* out) {
  const int ch = blockIdx.y * 256 + threadIdx.x;
  if (ch * 8 >= H) return;
  for (long long t = blockIdx.x; t < T; t += gridDim.x) {
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (residual) unpack8(*reinterpret_cast<const uint4*>(residual + t * H + ch * 8), acc);
    for (int j0 = 0; j0 < k; j0 += kCombineRows) {
      uint4 v[kCombineRows];
      float w[kCombineRows];
      bool there[kCombineRows];
#pragma unroll
      for (int j = 0; j < kCombineRows; ++j) {
        const int r = j0 + j < k ? dst[t * k + j0 + j] : -1;
        there[j] = r >= 0 && r < M_cap;
        if (!there[j]) continue;
        w[j] = weights ? weights[t * k + j0 + j] : 1.0f;
        v[j] = *reinterpret_cast<const uint4*>(y + (long long)r * H + ch * 8);
      }
#pragma unroll
      for (int j = 0; j < kCombineRows; ++j) {
        if (!there[j]) continue;
        float f[8];
        unpack8(v[j], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] = fmaf(w[j], f[q], acc[q]);
      }
    }
    *reinterpret_cast<uint4*>(out + t * H + ch * 8) = pack8(acc);
  }
}

// dy[dst[t][j]] = w[t][j] dout[t] and dweights[t][j] = <dout[t], y[dst[t][j]]>.
// One workgroup per token.  A row that stands twice among a token's slots
// gets the sum of their weights, written once.
__global__ __launch_bounds__(256) void combine_bwd_kernel(const uint16_t* __restrict__ dout,
                                                          const uint16_t* __restrict__ y, int M_cap, int H,
                                                          const int* __restrict__ dst,
                                                          const float* __restrict__ weights, int T, int k,
                                                          uint16_t* __restrict__ dy,
                                                          float* __restrict__ dweights) {
  __shared__ int row_s[kMaxTopk];
  __shared__ float w_s[kMaxTopk];
  __shared__ float part[4][kMaxTopk];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (long long t = blockIdx.x; t < T; t += gridDim.x) {
    __syncthreads();
    if ((int)threadIdx.x < k) {
      const int j = threadIdx.x;
      const int r = dst[t * k + j];
      bool first = true;
      float w = 0.0f;
      for (int i = 0; i < k; ++i)
        if (dst[t * k + i] == r) {
          if (i < j) first = false;
          w += weights ? weights[t * k + i] : 1.0f;
        }
      row_s[j] = r < 0 || r >= M_cap ? -1 : (first ? r : r | (int)0x80000000);   // top bit: not written
      w_s[j] = w;
    }
    __syncthreads();
    float dot[kMaxTopk];
#pragma unroll
    for (int j = 0; j < kMaxTopk; ++j) dot[j] = 0.0f;
    for (int ch = threadIdx.x; ch * 8 < H; ch += 256) {
      float d[8];
      unpack8(*reinterpret_cast<const uint4*>(dout + t * H + ch * 8), d);
#pragma unroll
      for (int j = 0; j < kMaxTopk; ++j) {
        if (j >= k) break;
        const int rs = row_s[j];
        if (rs == -1) continue;
        const long long at = (long long)(rs & 0x7FFFFFFF) * H + ch * 8;
        if (dweights) {
          float v[8];
          unpack8(*reinterpret_cast<const uint4*>(y + at), v);
#pragma unroll
          for (int q = 0; q < 8; ++q) dot[j] = fmaf(d[q], v[q], dot[j]);
        }
        if (dy && rs >= 0) {
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = w_s[j] * d[q];
          *reinterpret_cast<uint4*>(dy + at) = pack8(v);
        }
      }
    }
    if (dweights) {
#pragma unroll
      for (int j = 0; j < kMaxTopk; ++j) {
        if (j >= k) break;
        const float s = wave_sum(dot[j]);
        if (lane == 0) part[wave][j] = s;
      }
      __syncthreads();
      if ((int)threadIdx.x < k) {
        const int j = threadIdx.x;
        dweights[t * k + j] = part[0][j] + part[1][j] + part[2][j] + part[3][j];
      }
    }
  }
}

// ---------------------------------------------------------------- add + RMS norm
// Sum over the workgroup's NW waves; every thread gets it.  The partial sums
// are added in wave order.
template <int NW, class V>
__device__ __forceinline__ V block_sum(V v, V* tmp) {
  v = wave_sum(v);
  if constexpr (NW == 1) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  V s = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += tmp[w];
  return s;
}

// v (rh + rl) w rounded to a float once: v rh in two floats, and what they and rl
// leave added to their product with w.  Three roundings, of 1 / sqrt and of two
// products, would put one value in 10^5 on the other side of its rounding to
// bf16, and with it the scale of a block whose largest it is.  A zero keeps its
// sign, and where a part is not finite the plain product stays.
__device__ __forceinline__ float norm_value(float v, float rh, float rl, float w) {
#pragma clang fp contract(off)
  const float p = v * rh;
  const float e = fmaf(v, rl, fmaf(v, rh, -p));
  const float t = fmaf(p, w, e * w);
  return fabsf(t) > 0.0f ? t : p * w;
}

// One workgroup of NT threads per row, NC chunks of 8 columns per thread.
// h = bf16(x + residual) is what the residual stream keeps and what the norm
// is taken of, so that the backward pass sees the same values; y is rounded
// once, and the MXFP8 copy is the rounded y's (as the GEMM epilogues do).
// The row's sum is kept in 64 bits over chunks of 8 squares (exact in 32 bits
// but for their additions), 1 / sqrt in two floats (norm_value), at no cost in
// time while six waves per SIMD fit (five: 3% slower).
// Bound by memory: 16384 x 7168 with residual and MXFP8 copy 0.20 ms, 5.3 TB/s,
// the rate of a large copy; one row is one round trip to memory (the weights
// are fetched with the row) and a workgroup-wide sum.
template <int NT, int NC>
__global__ __launch_bounds__(NT, NT == 1024 ? 4 : NC <= 4 ? 6 : 4) void add_rmsnorm_kernel(NormArgs p) {
  __shared__ double tmp[NT / 64];
  constexpr bool kEarly = NT == 1024;
  const int nch = p.H >> 3;
  for (long long r = blockIdx.x; r < p.T; r += gridDim.x) {
    uint4 wt[NC];
    float v[NC][8];
    double sq = 0.0;   // of chunks' sums
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int ch = c * NT + threadIdx.x;
      if (ch >= nch) continue;
      const long long at = r * p.H + ch * 8;
      if (kEarly) wt[c] = *reinterpret_cast<const uint4*>(p.weight + ch * 8);
      unpack8(*reinterpret_cast<const uint4*>(p.x + at), v[c]);
      if (p.residual) {
        float w[8];
        unpack8(*reinterpret_cast<const uint4*>(p.residual + at), w);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[c][q] += w[q];
        const uint4 hv = pack8(v[c]);
        if (p.h) *reinterpret_cast<uint4*>(p.h + at) = hv;
        unpack8(hv, v[c]);
      } else if (p.h) {
        *reinterpret_cast<uint4*>(p.h + at) = pack8(v[c]);
      }
      float s8 = 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) s8 = fmaf(v[c][q], v[c][q], s8);
      sq += (double)s8;
    }
    double mean = block_sum<NT / 64>(sq, tmp) * p.inv_h + (double)p.eps;
    float m32 = (float)mean;
    double unit = 1.0;
    if (!(m32 > 1e-30f && m32 < 1e30f)) {   // (the whole workgroup)
      // squares that pass fp32's range: the sum again of values in another unit,
      // which small values keep below
      const bool small = m32 < 1.0f;
      const float u = small ? 0x1p100f : 0x1p-70f;
      sq = 0.0;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (c * NT + (int)threadIdx.x >= nch) continue;
        float s8 = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float t = v[c][q] * u;
          s8 = fmaf(t, t, s8);
          v[c][q] = small ? t : v[c][q];
        }
        sq += (double)s8;
      }
      unit = (double)u;
      mean = block_sum<NT / 64>(sq, tmp) * p.inv_h + (double)p.eps * unit * unit;
      m32 = (float)mean;
    }
    // 1 / sqrt in 32 bits and one Newton step in 64
    double rd = (double)(1.0f / sqrtf(m32));
    if (m32 > 0.0f && m32 < INFINITY) rd = rd * (1.5 - 0.5 * mean * rd * rd);
    const float rstd = (float)(rd * unit);
    if (unit < 1.0) rd *= unit;
    const float rh = (float)rd, rlow = rd < (double)INFINITY ? (float)(rd - (double)rh) : 0.0f;
    if (p.rstd && threadIdx.x == 0) p.rstd[r] = rstd;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int ch = c * NT + threadIdx.x;
      if (ch >= nch) continue;   // (with p.q a row is whole blocks of 4 lanes)
      const long long at = r * p.H + ch * 8;
      float w[8];
      unpack8(kEarly ? wt[c] : *reinterpret_cast<const uint4*>(p.weight + ch * 8), w);
#pragma unroll
      for (int q = 0; q < 8; ++q) w[q] = norm_value(v[c][q], rh, rlow, w[q]);
      const uint4 yv = pack8(w);
      if (p.y) *reinterpret_cast<uint4*>(p.y + at) = yv;
      if (p.q) {
        unpack8(yv, w);
        float amax = 0.0f;
        int nan = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          amax = fmaxf(amax, fabsf(w[q]));
          nan |= w[q] != w[q];
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          amax = fmaxf(amax, __shfl_xor(amax, d, 64));
          nan |= __shfl_xor(nan, d, 64);
        }
        const int E = nan ? 128 : mx_scale_exponent(amax, p.e5 ? 15 : 8);
        uint32_t lo = 0x7F7F7F7Fu, hi = 0x7F7F7F7Fu;
        if (E != 128) {
#pragma unroll
          for (int q = 0; q < 8; ++q) w[q] = ldexpf(w[q], -E);
          lo = p.e5 ? e5m2x4(w[0], w[1], w[2], w[3]) : e4m3x4(w[0], w[1], w[2], w[3]);
          hi = p.e5 ? e5m2x4(w[4], w[5], w[6], w[7]) : e4m3x4(w[4], w[5], w[6], w[7]);
        }
        // (row_q may have any alignment)
        uint8_t* q8 = p.q + at;
        if ((reinterpret_cast<uintptr_t>(p.q) & 7) == 0) {
          *reinterpret_cast<uint2*>(q8) = make_uint2(lo, hi);
        } else {
          for (int i = 0; i < 4; ++i) {
            q8[i] = (uint8_t)(lo >> (8 * i));
            q8[4 + i] = (uint8_t)(hi >> (8 * i));
          }
        }
        if ((threadIdx.x & 3) == 0) p.s[(r * p.H >> 5) + (ch >> 2)] = e8m0_byte(E);
      }
    }
  }
}

// With n = h rstd and g = dy weight: dx = rstd (g - n mean(g n)) + dh, and
// dweight = sum over rows of dy n.  Each workgroup takes rows blockIdx.x +
// i gridDim.x, the next one's loads going out before the current one's sum, and
// keeps its columns' share of dweight in registers; the shares are added in a
// fixed order by the kernel below.  Bound by memory.
template <int NC>
__global__ __launch_bounds__(256) void add_rmsnorm_bwd_kernel(NormBwdArgs p) {
  __shared__ float tmp[4];
  const int nch = p.H >> 3;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float dwt[NC][8], w[NC][8];
  uint4 dy[NC], h[NC], dh[NC];
  float rstd = 0.0f;
  auto fetch = [&](long long r) {
    rstd = p.rstd[r];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int ch = c * 256 + threadIdx.x;
      dy[c] = h[c] = dh[c] = zero;
      if (ch >= nch) continue;
      const long long at = r * p.H + ch * 8;
      dy[c] = *reinterpret_cast<const uint4*>(p.dy + at);
      h[c] = *reinterpret_cast<const uint4*>(p.h + at);
      if (p.dx && p.dh) dh[c] = *reinterpret_cast<const uint4*>(p.dh + at);
    }
  };
  if (blockIdx.x < p.T) fetch(blockIdx.x);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int ch = c * 256 + threadIdx.x;
    unpack8(ch < nch ? *reinterpret_cast<const uint4*>(p.weight + ch * 8) : zero, w[c]);
#pragma unroll
    for (int q = 0; q < 8; ++q) dwt[c][q] = 0.0f;
  }
  for (long long r = blockIdx.x; r < p.T; r += gridDim.x) {
    float n[NC][8], g[NC][8], d[NC][8];
    const float rs = rstd;
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      unpack8(dy[c], g[c]);
      unpack8(h[c], n[c]);
      unpack8(dh[c], d[c]);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        n[c][q] *= rs;
        dwt[c][q] = fmaf(g[c][q], n[c][q], dwt[c][q]);
        g[c][q] *= w[c][q];
        dot = fmaf(g[c][q], n[c][q], dot);
      }
    }
    if (r + gridDim.x < p.T) fetch(r + gridDim.x);
    if (!p.dx) continue;
    const float mean = block_sum<4>(dot, tmp) / (float)p.H;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int ch = c * 256 + threadIdx.x;
      if (ch >= nch) continue;
#pragma unroll
      for (int q = 0; q < 8; ++q) d[c][q] += rs * (g[c][q] - n[c][q] * mean);
      *reinterpret_cast<uint4*>(p.dx + r * p.H + ch * 8) = pack8(d[c]);
    }
  }
  if (p.part) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int ch = c * 256 + threadIdx.x;
      if (ch >= nch) continue;
      float4* o = reinterpret_cast<float4*>(p.part + (long long)blockIdx.x * p.H + ch * 8);
      o[0] = make_float4(dwt[c][0], dwt[c][1], dwt[c][2], dwt[c][3]);
      o[1] = make_float4(dwt[c][4], dwt[c][5], dwt[c][6], dwt[c][7]);
    }
  }
}

// dweight (+)= the sum of nparts partial rows, in a fixed order: a workgroup
// takes 32 columns (8 threads of 4), thread group g of 32 the rows g, g + 32,
// ..., whose sums are then added in order of g.
__global__ __launch_bounds__(256) void norm_dweight_kernel(const float* __restrict__ part, int nparts,
                                                           int H, float* __restrict__ dweight,
                                                           int accumulate) {
  __shared__ float4 sums[32][8];
  const int cl = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + cl * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < H) {   // (H is a multiple of 8)
#pragma unroll 8
    for (int i = g; i < nparts; i += 32) {
      const float4 v = *reinterpret_cast<const float4*>(part + (long long)i * H + col);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  sums[g][cl] = s;
  __syncthreads();
  if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < H) {
    const int c = threadIdx.x;
    float* o = dweight + blockIdx.x * 32 + c;
    float t = accumulate ? *o : 0.0f;
    for (int i = 0; i < 32; ++i) t += reinterpret_cast<const float*>(&sums[i][c >> 2])[c & 3];
    *o = t;
  }
}

}  // namespace moe
