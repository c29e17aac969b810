// AdamW over many tensors in one launch per width of state, its 8-bit states, and the
// norm of all gradients.  Each element's parameter, master, gradient and states are read and
// written once: the kernels are bound by memory.
//
// A table on the device lists chunks of 4096 elements of the tensors (2048 where there
// are few), each with all that its workgroup needs, so that one load leads to the
// elements however many tensors there are.  A thread takes four consecutive elements of
// each 1024: 16 bytes of fp32, 8 of bf16, 4 of 8-bit codes.
#pragma once

#include "device_common.hpp"
#include "operator_args.hpp"

namespace moe {

struct AdamwHyper {
  float beta1, rest1, c1, beta2, rest2, c2, eps, step_size, root_scale, decay, grad_scale;
  bool exact_root;             // an eps so small that roots of denormals count (1.1e-19 at most: 2^-26 of 1e-11)
  double beta1d, c1d, beta2d, c2d;   // 64-bit forms; c1d and c2d take the gradient's factor in
};

template <bool BF16>
__device__ __forceinline__ void load4(const void* p, long long i, int n, float* v) {
  if (n == 4) {
    if constexpr (BF16) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
      v[0] = __uint_as_float(w.x << 16);
      v[1] = __uint_as_float(w.x & 0xFFFF0000u);
      v[2] = __uint_as_float(w.y << 16);
      v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
      const f32x4 w = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
      v[0] = w[0]; v[1] = w[1]; v[2] = w[2]; v[3] = w[3];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = 0.0f;
      if (k < n) {
        if constexpr (BF16) v[k] = bf16_to_f32(static_cast<const uint16_t*>(p)[i + k]);
        else v[k] = static_cast<const float*>(p)[i + k];
      }
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, long long i, int n, const float* v) {
  if (n == 4) {
    if constexpr (BF16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else
      *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i) = f32x4{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) {
        if constexpr (BF16) static_cast<uint16_t*>(p)[i + k] = f32_to_bf16(v[k]);
        else static_cast<float*>(p)[i + k] = v[k];
      }
  }
}
__device__ __forceinline__ uint32_t load_codes4(const void* p, long long i, int n) {
  if (n == 4) return *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p) + i);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) w |= (uint32_t) static_cast<const uint8_t*>(p)[i + k] << (8 * k);
  return w;
}
__device__ __forceinline__ void store_codes4(void* p, long long i, int n, uint32_t w) {
  if (n == 4) {
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + i) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) static_cast<uint8_t*>(p)[i + k] = (uint8_t)(w >> (8 * k));
}

// ---------------------------------------------------------------- 8-bit states
// A block of 128 elements (32 lanes) shares m_scale = max |m| and v_scale =
// sqrt(max v), in fp32 (a power of two would round a block's slow decay away):
//   m = sign(c) (c / 127)^2 m_scale        c int8
//   sqrt(v) = (c / 255)^2 v_scale          c uint8, at least 1 for v > 0
// The square spreads the codes: a step is 1.6% of the block's largest value near
// it and still 16% at a hundredth of it.  An element's second moment never
// becomes 0 beside a first that did not.  With beta2 above 0.9922 no step without
// a gradient is half a code: an element's v then falls with its block's scale alone.
// The code is the nearest under the square root (the lower of two as near) as 64
// bits decide it: it is found in 32 bits, and only where they come near a border (or
// their range ends) compared with it in 64.
__device__ __forceinline__ double m_of_code(int c, double scale) {
  return (double)(c * (c < 0 ? -c : c)) * (1.0 / 16129.0) * scale;
}
__device__ __forceinline__ double root_of_code(int c, double scale) { return (double)(c * c) * (1.0 / 65025.0) * scale; }

__device__ __forceinline__ int code_m_exact(double a, double scale) {   // a = |m|, scale > 0
  int c = (int)rint(127.0 * sqrt(a / scale));
  c = c > 127 ? 127 : c;
  const double t = a * 64516.0;                 // 4 * 127^2
  const int up = 2 * c + 1, down = 2 * c - 1;
  if (t > (double)(up * up) * scale) ++c;
  else if (c > 0 && t <= (double)(down * down) * scale) --c;
  return c > 127 ? 127 : c;
}
__device__ __forceinline__ int code_root_exact(double v, double scale) {
  int c = (int)rint(255.0 * sqrt(sqrt(v) / scale));
  c = c > 255 ? 255 : c;
  const double t = v * 67652010000.0, s2 = scale * scale;   // 510^4
  const double up = (double)((2 * c + 1) * (2 * c + 1)), down = (double)((2 * c - 1) * (2 * c - 1));
  if (t > up * up * s2) ++c;
  else if (c > 0 && t <= down * down * s2) --c;
  return c > 255 ? 255 : c;
}
// With u = 2^-24: m, 1 / m_scale (2 u) and their product make the ratio in x = 127
// sqrt(m / m_scale) right to 4 u, the hardware's root (2 u) and the product x to 5 u;
// v, its block's largest (1 u each), the reciprocal, the product and v_scale's rounding
// (2 u) make the ratio in y = 255 sqrt(sqrt(v) / v_scale) right to 7 u, two roots and the
// product y to 6 u.  Nearer than that to the middle between two codes, 127 * 5 u = 3.8e-5
// and 255 * 6 u = 9.2e-5, the 64-bit comparison decides.
__device__ __forceinline__ bool near_border(float x, float near) {
  return fabsf(fabsf(x - rintf(x)) - 0.5f) < near;
}
constexpr float kNearM = 5e-5f, kNearRoot = 1.2e-4f;

// over the 32 lanes of a block: rotations within 16 lanes, then the other 16
template <int CTRL>
__device__ __forceinline__ uint32_t rotate(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ float half_max(float v) {
  v = fmaxf(v, __uint_as_float(rotate<0x128>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(rotate<0x124>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(rotate<0x122>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(rotate<0x121>(__float_as_uint(v))));
  return fmaxf(v, __shfl_xor(v, 16, 64));
}
template <int CTRL>
__device__ __forceinline__ double max_rotated(double v) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
  const unsigned long long o = (unsigned long long)rotate<CTRL>((uint32_t)(b >> 32)) << 32 | rotate<CTRL>((uint32_t)b);
  return fmax(v, __builtin_bit_cast(double, o));
}
__device__ __forceinline__ double half_max(double v) {
  v = max_rotated<0x128>(v);
  v = max_rotated<0x124>(v);
  v = max_rotated<0x122>(v);
  v = max_rotated<0x121>(v);
  return fmax(v, __shfl_xor(v, 16, 64));
}
// fp32 of the square root of a 64-bit value
__device__ __forceinline__ float root_of(double v) {
  if (!(v > 1e-30 && v < 1e30)) return (float)sqrt(v);
  // a 1-ulp root and the middles between it and its neighbours, whose squares have
  // 50 bits
  const float s = __builtin_amdgcn_sqrtf((float)v);
  const float up = __uint_as_float(__float_as_uint(s) + 1), down = __uint_as_float(__float_as_uint(s) - 1);
  const double mu = 0.5 * ((double)s + (double)up), md = 0.5 * ((double)s + (double)down);
  return v > mu * mu ? up : v < md * md ? down : s;
}

// Four elements of a thread, as memory holds them.  PARAM: 0 fp32, 1 bf16, 2 bf16
// with an fp32 master.
template <bool STATE8>
struct AdamwFour {
  float g[4], p[4], m[4], v[4];
};
template <>
struct AdamwFour<true> {
  float g[4], p[4], m_scale, v_scale;
  uint32_t m, v;
};
// fp32's largest value for an infinity: what a small correction of a value takes, so
// that an infinite one stays as it is (a NaN is in the value itself).
__device__ __forceinline__ float finite_of(float v) {
  return __builtin_amdgcn_fmed3f(v, -3.402823466e38f, 3.402823466e38f);
}
// elements i .. i + n of the tensor, n <= 4 (WHOLE: n = 4, with nothing skipped, so
// that the compiler can count the loads on their way)
template <int PARAM, bool GRAD16, bool STATE8, bool WHOLE>
__device__ __forceinline__ void adamw_load(const AdamwChunk& t, int i, int n, AdamwFour<STATE8>& f) {
  if constexpr (WHOLE) n = 4;
  load4<GRAD16>(t.grad, i, n, f.g);
  if constexpr (PARAM == 1) load4<true>(t.param, i, n, f.p);
  else load4<false>(PARAM == 2 ? t.master : t.param, i, n, f.p);
  if constexpr (STATE8) {
    f.m = load_codes4(t.m, i, n);
    f.v = load_codes4(t.v, i, n);
    f.m_scale = n > 0 ? t.m_scale[i / kAdamwBlock] : 0.0f;
    f.v_scale = n > 0 ? t.v_scale[i / kAdamwBlock] : 0.0f;
  } else {
    load4<false>(t.m, i, n, f.m);
    load4<false>(t.v, i, n, f.v);
  }
}
template <int PARAM, bool STATE8, bool WHOLE>
__device__ __forceinline__ void adamw_update(const AdamwChunk& t, int i, int n, const AdamwHyper& h,
                                             const AdamwFour<STATE8>& f) {
  if constexpr (WHOLE) n = 4;
  float m[4], v[4], p[4];
  if constexpr (!STATE8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float gk = f.g[k] * h.grad_scale;
      // beta in two parts: fp32's alone is off by up to 2^-25, so that it and 1 - beta do not
      // add up to 1 (beta2 = 0.99999: v settles 0.14% off; 1 - 2e-8: it is 1, v only grows).
      m[k] = fmaf(h.beta1, f.m[k], fmaf(h.rest1, finite_of(f.m[k]), h.c1 * gk));
      v[k] = fmaf(h.beta2, f.v[k], fmaf(h.rest2, finite_of(f.v[k]), h.c2 * (gk * gk)));
    }
    store4<false>(t.m, i, n, m);
    store4<false>(t.v, i, n, v);
  } else {
    const double ms = f.m_scale, vs = f.v_scale;
    const double km = h.beta1d * (1.0 / 16129.0) * ms, kv = h.beta2d * (1.0 / (65025.0 * 65025.0)) * vs * vs;
    double md[4], vd[4];
    float ma = 0.0f;
    double va = 0.0;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = (int)(int8_t)(f.m >> (8 * k)), d = (int)(f.v >> (8 * k) & 0xFF);
      const double gk = (double)f.g[k], d2 = (double)(d * d);
      md[k] = (double)(c * (c < 0 ? -c : c)) * km + gk * h.c1d;
      vd[k] = d2 * d2 * kv + gk * gk * h.c2d;
      if (!WHOLE && k >= n) md[k] = vd[k] = 0.0;
      m[k] = (float)md[k];
      v[k] = (float)vd[k];
      ma = fmaxf(ma, fabsf(m[k]));
      va = fmax(va, vd[k]);
    }
    // sums of sizes, which a NaN or an infinity (or values near fp32's end) leave
    if (!((fabsf(m[0]) + fabsf(m[1])) + (fabsf(m[2]) + fabsf(m[3])) < INFINITY) ||
        !((vd[0] + vd[1]) + (vd[2] + vd[3]) < (double)INFINITY))
#pragma unroll
      for (int k = 0; k < 4; ++k) bad = bad || !(fabsf(m[k]) < INFINITY) || !(vd[k] < (double)INFINITY);
    ma = half_max(ma);
    va = half_max(va);
    const float root_max = root_of(va);
    const unsigned long long any = __ballot(bad || !(root_max < INFINITY));
    const bool lost = (threadIdx.x & 32 ? any >> 32 : any & 0xFFFFFFFFull) != 0;
    // a NaN or an infinity leaves no codes: the block's states are NaN from here
    const float m_scale = lost ? __uint_as_float(0x7FC00000u) : ma;
    const float v_scale = lost ? __uint_as_float(0x7FC00000u) : root_max;
    // outside of these the ratios below leave the normal numbers of 32 bits
    const bool m_in = ma > 1e-25f && ma < 1e30f, v_in = va > 1e-25 && va < 1e30;
    const float im = __builtin_amdgcn_rcpf(ma), iv = __builtin_amdgcn_rcpf((float)va);
    float x[4], y[4];
    int om[4], ov[4];
    bool unsure = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = fminf(127.0f * __builtin_amdgcn_sqrtf(fabsf(m[k]) * im), 127.0f);
      y[k] = fminf(255.0f * __builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(v[k] * iv)), 255.0f);
      unsure = unsure || near_border(x[k], kNearM) || near_border(y[k], kNearRoot);
      om[k] = (int)rintf(x[k]);
      ov[k] = (int)rintf(y[k]);
    }
    if (!m_in || !v_in) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        om[k] = m_scale > 0.0f ? code_m_exact(fabs(md[k]), (double)m_scale) : 0;
        ov[k] = v_scale > 0.0f ? code_root_exact(vd[k], (double)v_scale) : 0;
      }
    } else if (unsure) {
      // above the middle between floor and the code after it?
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = (int)x[k], d = (int)y[k];
        om[k] = c + (fabs(md[k]) * 64516.0 > (double)((2 * c + 1) * (2 * c + 1)) * (double)m_scale);
        const double d2 = (double)((2 * d + 1) * (2 * d + 1));
        ov[k] = d + (vd[k] * 67652010000.0 > d2 * d2 * ((double)v_scale * (double)v_scale));
        om[k] = min(om[k], 127);
        ov[k] = min(ov[k], 255);
      }
    }
    uint32_t wm = 0, wv = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = lost ? 0 : md[k] < 0.0 ? -om[k] : om[k];
      const int d = lost || !(v_scale > 0.0f) ? 0 : vd[k] > 0.0 ? max(ov[k], 1) : 0;
      wm |= (uint32_t)(c & 0xFF) << (8 * k);
      wv |= (uint32_t)d << (8 * k);
    }
    store_codes4(t.m, i, n, wm);
    store_codes4(t.v, i, n, wv);
    if ((threadIdx.x & 31) == 0 && n > 0) {
      t.m_scale[i / kAdamwBlock] = m_scale;
      t.v_scale[i / kAdamwBlock] = v_scale;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float w = v[k] * h.root_scale;
    // the hardware's root and reciprocal, 1 ulp each; they flush denormals, which
    // matter beside an eps near 0 alone
    const float update = h.exact_root ? m[k] * h.step_size / (sqrtf(w) + h.eps)
                                      : m[k] * h.step_size * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(w) + h.eps);
    // (p times fp32's 1 - lr decay would round every element's decay the same way, to a
    // multiple of 2^-24: lr decay = 1e-7 acted as 1.19e-7, below 3e-8 as 0)
    p[k] = f.p[k] - fmaf(h.decay, finite_of(f.p[k]), update);
  }
  if constexpr (PARAM == 2) store4<false>(t.master, i, n, p);
  if constexpr (PARAM == 0) store4<false>(t.param, i, n, p);
  else store4<true>(t.param, i, n, p);
}

// One chunk: its whole steps two at a time, their loads together, then what is left.
template <int PARAM, bool GRAD16, bool STATE8>
__device__ __forceinline__ void adamw_chunk(const AdamwChunk& t, const AdamwHyper& h) {
  constexpr int STEPS = 2;
  const int i = 4 * threadIdx.x;
  int at = 0;
  for (; at + STEPS * kAdamwStep <= t.n; at += STEPS * kAdamwStep) {
    AdamwFour<STATE8> f[STEPS];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) adamw_load<PARAM, GRAD16, STATE8, true>(t, at + i + kAdamwStep * k, 4, f[k]);
#pragma unroll
    for (int k = 0; k < STEPS; ++k) adamw_update<PARAM, STATE8, true>(t, at + i + kAdamwStep * k, 4, h, f[k]);
  }
  for (; at < t.n; at += kAdamwStep) {
    const int n = max(0, min(4, t.n - at - i));
    AdamwFour<STATE8> f;
    adamw_load<PARAM, GRAD16, STATE8, false>(t, at + i, n, f);
    adamw_update<PARAM, STATE8, false>(t, at + i, n, h, f);
  }
}

// m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2, p' = p - (lr decay p + lr
// (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps)).  The chunks of 32-bit and of
// 8-bit states lie apart, each with a kernel of its own.  Measured, bf16 parameters with
// masters and fp32 gradients: 531M elements of 32-bit states 3.15 ms, 5.1 TB/s; 265M of 8-bit
// ones 0.99 ms, 4.8 TB/s; 1.1M in 16 tensors 6 us.
template <bool STATE8>
__global__ __launch_bounds__(256, 4) void adamw_kernel(AdamwArgs a, const AdamwChunk* __restrict__ chunks,
                                                    long long first_chunk, long long end_chunk) {
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  if (gs != gs) return;                        // gradients without a norm: no step
  const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
  double bias1 = a.bias1, bias2 = a.bias2;
  if (a.step) {
    const int t = *a.step < 1 ? 1 : *a.step;
    bias1 = 1.0 - pow(a.beta1, (double)t);
    bias2 = 1.0 - pow(a.beta2, (double)t);
  }
  AdamwHyper h;
  h.beta1d = a.beta1;
  h.c1d = (1.0 - a.beta1) * (double)gs;
  h.beta2d = a.beta2;
  h.c2d = (1.0 - a.beta2) * (double)gs * (double)gs;
  h.beta1 = (float)a.beta1;
  h.rest1 = (float)(a.beta1 - (double)h.beta1);
  h.c1 = (float)(1.0 - a.beta1);
  h.beta2 = (float)a.beta2;
  h.rest2 = (float)(a.beta2 - (double)h.beta2);
  h.c2 = (float)(1.0 - a.beta2);
  h.eps = (float)a.eps;
  h.exact_root = a.eps < 1e-11;
  h.root_scale = (float)(1.0 / bias2);
  h.grad_scale = gs;
  AdamwChunk next = chunks[first_chunk + blockIdx.x];   // (a workgroup has one chunk at least)
  for (long long c = first_chunk + blockIdx.x; c < end_chunk; c += gridDim.x) {
    const AdamwChunk t = next;
    next = chunks[min(c + gridDim.x, end_chunk - 1)];
    if (!t.param) continue;
    h.step_size = (float)(lr * (double)t.lr_scale / bias1);
    h.decay = (float)(lr * (double)t.lr_scale * (double)t.decay);
    if (t.grad_bf16) {
      if (t.master) adamw_chunk<2, true, STATE8>(t, h);
      else if (t.param_bf16) adamw_chunk<1, true, STATE8>(t, h);
      else adamw_chunk<0, true, STATE8>(t, h);
    } else {
      if (t.master) adamw_chunk<2, false, STATE8>(t, h);
      else if (t.param_bf16) adamw_chunk<1, false, STATE8>(t, h);
      else adamw_chunk<0, false, STATE8>(t, h);
    }
  }
}

// 8-bit states as fp32 (265M elements: 0.47 ms, 5.6 TB/s).
__global__ __launch_bounds__(256) void adamw_unpack_kernel(const int8_t* __restrict__ m, const float* __restrict__ m_scale,
                                                           const uint8_t* __restrict__ v,
                                                           const float* __restrict__ v_scale, long long n,
                                                           float* __restrict__ m_out, float* __restrict__ v_out) {
  for (long long i = 4 * ((long long)blockIdx.x * 256 + threadIdx.x); i < n; i += 1024LL * gridDim.x) {
    const int k = n - i < 4 ? (int)(n - i) : 4;
    const long long block = i / kAdamwBlock;
    if (m_out) {
      const uint32_t c = load_codes4(m, i, k);
      const double s = m_scale[block];
      float o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = (float)m_of_code((int)(int8_t)(c >> (8 * j)), s);
      store4<false>(m_out, i, k, o);
    }
    if (v_out) {
      const uint32_t c = load_codes4(v, i, k);
      const double s = v_scale[block];
      float o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double r = root_of_code((int)(c >> (8 * j) & 0xFF), s);
        o[j] = (float)(r * r);
      }
      store4<false>(v_out, i, k, o);
    }
  }
}

// ---------------------------------------------------------------- norm of the gradients
// Squares summed in 64 bits (their range too: the squares of fp32 values do not
// fit fp32), each workgroup over chunks in a fixed order.  Bound by reading: 265M fp32
// gradients 164 us, 6.5 TB/s; a second launch adds the workgroups' sums (one launch of
// many would need a counter that each call finds at 0).
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* tmp) {   // tmp: WAVES of LDS
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) v += tmp[w];
  return v;
}
// by 256 threads, of which this is the tid-th
template <bool BF16>
__device__ __forceinline__ void add_squares(const AdamwChunk& t, int tid, double* sum) {
  const auto add = [&](const float* g) {
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = fma((double)g[k], (double)g[k], sum[k]);
  };
  const int i = 4 * tid;
  int at = 0;
  for (; at + 2 * kAdamwStep <= t.n; at += 2 * kAdamwStep) {
    float g[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) load4<BF16>(t.grad, at + kAdamwStep * s + i, 4, g[s]);
#pragma unroll
    for (int s = 0; s < 2; ++s) add(g[s]);
  }
  for (; at < t.n; at += kAdamwStep) {
    float g[4];
    load4<BF16>(t.grad, at + i, max(0, min(4, t.n - at - i)), g);
    add(g);
  }
}
// chunks first, first + step, .. below n_chunks, the next one's table entry on its way
__device__ __forceinline__ double squares_of(const AdamwChunk* __restrict__ chunks, long long first, long long step,
                                             long long n_chunks, int tid) {
  double sum[4] = {};
  AdamwChunk next = chunks[min(first, n_chunks - 1)];
  for (long long c = first; c < n_chunks; c += step) {
    const AdamwChunk t = next;
    next = chunks[min(c + step, n_chunks - 1)];
    if (t.grad_bf16) add_squares<true>(t, tid, sum);
    else add_squares<false>(t, tid, sum);
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}
// out[0] = the norm, out[1] = min(1, max_norm / (norm + 1e-6)), NaN where the
// norm is not finite.
__device__ __forceinline__ void norm_out(double sum, float max_norm, float* out) {
  const double norm = sqrt(sum);
  const double f = (double)max_norm / (norm + 1e-6);
  const float n32 = (float)norm;
  out[0] = n32;
  out[1] = n32 < INFINITY ? (f > 1.0 ? 1.0f : (float)f) : __uint_as_float(0x7FC00000u);
}
__global__ __launch_bounds__(256) void grad_norm_kernel(const AdamwChunk* __restrict__ chunks, long long n_chunks,
                                                        double* __restrict__ part) {
  __shared__ double tmp[4];
  const double s = block_sum<4>(squares_of(chunks, blockIdx.x, gridDim.x, n_chunks, threadIdx.x), tmp);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}
__global__ __launch_bounds__(256) void grad_norm_final_kernel(const double* __restrict__ part, int parts,
                                                              float max_norm, float* __restrict__ out) {
  __shared__ double tmp[4];
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) sum += part[i];
  sum = block_sum<4>(sum, tmp);
  if (threadIdx.x == 0) norm_out(sum, max_norm, out);
}
// A plan of few chunks in one launch, four of them at a time.
__global__ __launch_bounds__(1024) void grad_norm_few_kernel(const AdamwChunk* __restrict__ chunks, long long n_chunks,
                                                             float max_norm, float* __restrict__ out) {
  __shared__ double tmp[16];
  const double s = n_chunks > 0 ? squares_of(chunks, threadIdx.x >> 8, 4, n_chunks, threadIdx.x & 255) : 0.0;
  const double sum = block_sum<16>(s, tmp);
  if (threadIdx.x == 0) norm_out(sum, max_norm, out);
}

}  // namespace moe
