// AdamW over many tensors in one launch, its 8-bit states, and the norm of all
// gradients.  Each element's parameter, master, gradient and states are read and
// written once: the kernels are bound by memory.
//
// A table on the device lists the tensors and cuts them into chunks of 4096
// elements, so that a workgroup finds its elements with two dependent loads
// however many tensors there are.  A thread takes four consecutive elements of
// each 1024: 16 bytes of fp32, 8 of bf16, 4 of 8-bit codes.
#pragma once

#include "device_common.hpp"
#include "operator_args.hpp"

namespace moe {

struct AdamwHyper {
  float beta1, c1, beta2, c2, eps, step_size, root_scale, shrink;   // fp32 forms
  double beta1d, c1d, beta2d, c2d;
  float grad_scale;
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
// becomes 0 beside a first that did not.  The nearest code under the square root
// (the lower of two as near) is found in 32 bits and put right by comparing with
// its borders in 64, so it is the one that the definition gives.
__device__ __forceinline__ double m_of_code(int c, double scale) {
  return (double)(c * (c < 0 ? -c : c)) * (1.0 / 16129.0) * scale;
}
__device__ __forceinline__ double root_of_code(int c, double scale) { return (double)(c * c) * (1.0 / 65025.0) * scale; }

__device__ __forceinline__ int nearest_m(double a, double scale, float guess) {   // a = |m|
  int c = (int)rintf(127.0f * sqrtf(guess));
  c = c > 127 ? 127 : c;
  const double t = a * 64516.0;                 // 4 * 127^2
  const int up = 2 * c + 1, down = 2 * c - 1;
  if (t > (double)(up * up) * scale) ++c;
  else if (c > 0 && t <= (double)(down * down) * scale) --c;
  return c > 127 ? 127 : c;
}
__device__ __forceinline__ int nearest_root(double v, double scale, float guess) {
  int c = (int)rintf(255.0f * sqrtf(sqrtf(guess)));
  c = c > 255 ? 255 : c;
  const double t = v * 67652010000.0, s2 = scale * scale;   // 510^4
  const double up = (double)((2 * c + 1) * (2 * c + 1)), down = (double)((2 * c - 1) * (2 * c - 1));
  if (t > up * up * s2) ++c;
  else if (c > 0 && t <= down * down * s2) --c;
  c = c > 255 ? 255 : c;
  return c < 1 && v > 0.0 ? 1 : c;
}
// over the 32 lanes of a block
__device__ __forceinline__ double half_max(double v) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) v = fmax(v, __shfl_xor(v, d, 64));
  return v;
}

// One chunk.  PARAM: 0 fp32, 1 bf16, 2 bf16 with an fp32 master.
template <int PARAM, bool GRAD16, bool STATE8>
__device__ __forceinline__ void adamw_chunk(const AdamwTensor& t, long long first, const AdamwHyper& h) {
  const long long left = t.n - first;
#pragma unroll
  for (int s = 0; s < kAdamwChunk / 1024; ++s) {
    const long long at = 1024LL * s + 4 * threadIdx.x;
    if (1024LL * s >= left) break;              // the same for the whole workgroup
    const long long i = first + at;
    const int n = at >= left ? 0 : left - at < 4 ? (int)(left - at) : 4;
    float g[4], p[4], m[4], v[4];
    load4<GRAD16>(t.grad, i, n, g);
    if constexpr (PARAM == 1) load4<true>(t.param, i, n, p);
    else load4<false>(PARAM == 2 ? t.master : t.param, i, n, p);
    if constexpr (!STATE8) {
      load4<false>(t.m, i, n, m);
      load4<false>(t.v, i, n, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float gk = g[k] * h.grad_scale;
        m[k] = h.beta1 * m[k] + h.c1 * gk;
        v[k] = h.beta2 * v[k] + h.c2 * (gk * gk);
      }
      store4<false>(t.m, i, n, m);
      store4<false>(t.v, i, n, v);
    } else {
      const long long block = i / kAdamwBlock;
      const uint32_t cm = load_codes4(t.m, i, n), cv = load_codes4(t.v, i, n);
      const double ms = n ? t.m_scale[block] : 0.0f, vs = n ? t.v_scale[block] : 0.0f;
      double md[4], vd[4];
      double ma = 0.0, va = 0.0;
      bool bad = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const double gk = (double)g[k] * (double)h.grad_scale;
        const double root = root_of_code((int)(cv >> (8 * k) & 0xFF), vs);
        md[k] = h.beta1d * m_of_code((int)(int8_t)(cm >> (8 * k)), ms) + h.c1d * gk;
        vd[k] = h.beta2d * (root * root) + h.c2d * (gk * gk);
        if (k >= n) md[k] = vd[k] = 0.0;
        m[k] = (float)md[k];
        v[k] = (float)vd[k];
        ma = fmax(ma, fabs(md[k]));
        va = fmax(va, vd[k]);
        bad = bad || !(fabsf(m[k]) < INFINITY) || !(vd[k] < (double)INFINITY);
      }
      ma = half_max(ma);
      va = half_max(va);
      const float root_max = (float)sqrt(va);
      const unsigned long long any = __ballot(bad || !(root_max < INFINITY));
      const bool lost = (threadIdx.x & 32 ? any >> 32 : any & 0xFFFFFFFFull) != 0;
      // a NaN or an infinity leaves no codes: the block's states are NaN from here
      const float m_scale = lost ? __uint_as_float(0x7FC00000u) : (float)ma;
      const float v_scale = lost ? __uint_as_float(0x7FC00000u) : root_max;
      const double im = m_scale > 0.0f ? 1.0 / (double)m_scale : 0.0, iv = v_scale > 0.0f ? 1.0 / va : 0.0;
      uint32_t om = 0, ov = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        int c = m_scale > 0.0f ? nearest_m(fabs(md[k]), (double)m_scale, (float)(fabs(md[k]) * im)) : 0;
        c = md[k] < 0.0 ? -c : c;
        const int d = v_scale > 0.0f ? nearest_root(vd[k], (double)v_scale, (float)(vd[k] * iv)) : 0;
        om |= (uint32_t)(c & 0xFF) << (8 * k);
        ov |= (uint32_t)d << (8 * k);
      }
      store_codes4(t.m, i, n, om);
      store_codes4(t.v, i, n, ov);
      if ((threadIdx.x & 31) == 0 && n) {
        t.m_scale[block] = m_scale;
        t.v_scale[block] = v_scale;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float update = m[k] * h.step_size / (sqrtf(v[k] * h.root_scale) + h.eps);
      p[k] = p[k] * h.shrink - update;
    }
    if constexpr (PARAM == 2) store4<false>(t.master, i, n, p);
    if constexpr (PARAM == 0) store4<false>(t.param, i, n, p);
    else store4<true>(t.param, i, n, p);
  }
}

template <int PARAM>
__device__ __forceinline__ void adamw_chunk_of(const AdamwTensor& t, long long first, const AdamwHyper& h) {
  if (t.state8) {
    if (t.grad_bf16) adamw_chunk<PARAM, true, true>(t, first, h);
    else adamw_chunk<PARAM, false, true>(t, first, h);
  } else {
    if (t.grad_bf16) adamw_chunk<PARAM, true, false>(t, first, h);
    else adamw_chunk<PARAM, false, false>(t, first, h);
  }
}

// m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2, p' = p (1 - lr decay) - lr
// (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps).
__global__ __launch_bounds__(256) void adamw_kernel(AdamwArgs a) {
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
  h.c1d = 1.0 - a.beta1;
  h.beta2d = a.beta2;
  h.c2d = 1.0 - a.beta2;
  h.beta1 = (float)h.beta1d;
  h.c1 = (float)h.c1d;
  h.beta2 = (float)h.beta2d;
  h.c2 = (float)h.c2d;
  h.eps = (float)a.eps;
  h.root_scale = (float)(1.0 / bias2);
  h.grad_scale = gs;
  for (long long c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    const AdamwChunk ch = a.chunks[c];
    const AdamwTensor t = a.tensors[ch.tensor];
    if (!t.param) continue;
    h.step_size = (float)(lr * (double)t.lr_scale / bias1);
    h.shrink = (float)(1.0 - lr * (double)t.lr_scale * (double)t.decay);
    const long long first = (long long)ch.index * kAdamwChunk;
    if (t.master) adamw_chunk_of<2>(t, first, h);
    else if (t.param_bf16) adamw_chunk_of<1>(t, first, h);
    else adamw_chunk_of<0>(t, first, h);
  }
}

// 8-bit states as fp32.
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
// fit fp32), each workgroup over chunks in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* tmp) {   // tmp: 4 of LDS; the result in thread 0
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  return tmp[0] + tmp[1] + tmp[2] + tmp[3];
}
template <bool BF16>
__device__ __forceinline__ void add_squares(const AdamwTensor& t, long long first, double* sum) {
  const long long left = t.n - first;
#pragma unroll
  for (int s = 0; s < kAdamwChunk / 1024; ++s) {
    const long long at = 1024LL * s + 4 * threadIdx.x;
    const int n = at >= left ? 0 : left - at < 4 ? (int)(left - at) : 4;
    float g[4];
    load4<BF16>(t.grad, first + at, n, g);
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = fma((double)g[k], (double)g[k], sum[k]);
  }
}
__global__ __launch_bounds__(256) void grad_norm_kernel(const AdamwTensor* __restrict__ tensors,
                                                        const AdamwChunk* __restrict__ chunks, long long n_chunks,
                                                        double* __restrict__ part) {
  __shared__ double tmp[4];
  double sum[4] = {};
  for (long long c = blockIdx.x; c < n_chunks; c += gridDim.x) {
    const AdamwChunk ch = chunks[c];
    const AdamwTensor t = tensors[ch.tensor];
    const long long first = (long long)ch.index * kAdamwChunk;
    if (t.grad_bf16) add_squares<true>(t, first, sum);
    else add_squares<false>(t, first, sum);
  }
  const double s = block_sum((sum[0] + sum[1]) + (sum[2] + sum[3]), tmp);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}
// out[0] = the norm, out[1] = min(1, max_norm / (norm + 1e-6)), NaN where the
// norm is not finite.
__global__ __launch_bounds__(256) void grad_norm_final_kernel(const double* __restrict__ part, int parts,
                                                              float max_norm, float* __restrict__ out) {
  __shared__ double tmp[4];
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) sum += part[i];
  sum = block_sum(sum, tmp);
  if (threadIdx.x != 0) return;
  const double norm = sqrt(sum);
  const double f = (double)max_norm / (norm + 1e-6);
  const float n32 = (float)norm;
  out[0] = n32;
  out[1] = n32 < INFINITY ? (f > 1.0 ? 1.0f : (float)f) : __uint_as_float(0x7FC00000u);
}

}  // namespace moe
