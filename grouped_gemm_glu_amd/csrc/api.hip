// C ABI of the MoE GroupGEMM + GLU library: argument checking, the cached
// device properties and the launches.  Every entry point validates what the
// host can see and returns before any launch on error; nothing here
// allocates, synchronises or reads device memory back.
#include <math.h>
#include <string.h>

#include <initializer_list>

#include "aux_kernels.hpp"
#include "internal.hpp"

using namespace moe;

namespace {

constexpr int kMaxDevices = 64;
int g_num_cus[kMaxDevices];  // 0 = not initialised

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// A buffer of a call: n bytes from p on (a null pointer: none).
struct Buf {
  const void* p;
  size_t n;
};
bool share_bytes(const Buf& a, const Buf& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n && b.n && (x <= y ? y - x < a.n : x - y < b.n);
}
// Whether an output shares bytes with an input or with another output: the
// kernels read rows that other workgroups' outputs could have replaced.
bool overlap(std::initializer_list<Buf> outputs, std::initializer_list<Buf> inputs) {
  for (const Buf* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Buf& i : inputs)
      if (share_bytes(*o, i)) return true;
    for (const Buf* o2 = o + 1; o2 != outputs.end(); ++o2)
      if (share_bytes(*o, *o2)) return true;
  }
  return false;
}
// bytes of rows x cols elements of bits each
size_t bytes_of(long long rows, long long cols, int bits = 16) { return (size_t)rows * (size_t)cols * (size_t)bits / 8; }

moe_status_t ensure_init(int* cus) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_DEVICE;
  if (g_num_cus[dev] == 0) {
    moe_status_t st = moe_init(dev);
    if (st != MOE_OK) return st;
  }
  *cus = g_num_cus[dev];
  return MOE_OK;
}

moe_status_t check_groups(const moe_groups_t* g) {
  if (!g || !g->counts) return MOE_ERR_NULL;
  if (g->E < 1 || g->E > kMaxExperts || g->M_cap < 0) return MOE_ERR_SHAPE;
  if (!aligned4(g->counts) || (g->offsets_out && !aligned4(g->offsets_out)) ||
      (g->status_out && !aligned4(g->status_out)))
    return MOE_ERR_ALIGN;
  return MOE_OK;
}

moe_status_t check_mx(const moe_mx_out_t* mx) {
  if (!mx) return MOE_OK;
  if ((mx->row_q == nullptr) != (mx->row_s == nullptr)) return MOE_ERR_NULL;
  if ((mx->col_q == nullptr) != (mx->col_s == nullptr)) return MOE_ERR_NULL;
  if (mx->e5m2 != 0 && mx->e5m2 != 1) return MOE_ERR_UNSUPPORTED;
  if (mx->col_blocked != 0 && mx->col_blocked != 1) return MOE_ERR_UNSUPPORTED;
  if (mx->col_blocked && mx->col_q && !aligned16(mx->col_q)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

moe_status_t fill_epilogue(const moe_epilogue_t* ep, EpiParams* out) {
  if (!ep) return MOE_ERR_NULL;
  if (ep->act < MOE_ACT_SWIGLU || ep->act > MOE_ACT_SRELU) return MOE_ERR_UNSUPPORTED;
  if (ep->bias && !aligned16(ep->bias)) return MOE_ERR_ALIGN;
  if (ep->row_scale && !aligned4(ep->row_scale)) return MOE_ERR_ALIGN;
  if (isnan(ep->alpha) || isnan(ep->gate_lo) || isnan(ep->gate_hi) || isnan(ep->up_lo) ||
      isnan(ep->up_hi) || isnan(ep->up_offset))
    return MOE_ERR_SHAPE;
  out->act = ep->act;
  out->alpha = ep->alpha;
  out->gate_lo = ep->gate_lo;
  out->gate_hi = ep->gate_hi;
  out->up_lo = ep->up_lo;
  out->up_hi = ep->up_hi;
  out->up_offset = ep->up_offset;
  out->bias = static_cast<const uint16_t*>(ep->bias);
  out->row_scale = ep->row_scale;
  if (ep->amax_out && !aligned4(ep->amax_out)) return MOE_ERR_ALIGN;
  out->amax_out = ep->amax_out;
  out->rht_signs = ep->rht_signs & 0xFFFFu;
  if ((ep->dbias_out && !aligned4(ep->dbias_out)) || (ep->drow_scale_out && !aligned4(ep->drow_scale_out)))
    return MOE_ERR_ALIGN;
  out->dbias_out = ep->dbias_out;
  out->drs_out = ep->drow_scale_out;
  return MOE_OK;
}

void fill_groups(GemmArgs* a, const moe_groups_t* g) {
  a->counts = g->counts;
  a->E = g->E;
  a->M_cap = g->M_cap;
  a->offsets_out = g->offsets_out;
  a->status_out = g->status_out;
}

void fill_mx(GemmArgs* a, const moe_mx_out_t* mx, int cols, const moe_groups_t* g) {
  a->row_q = mx ? mx->row_q : nullptr;
  a->row_s = mx ? mx->row_s : nullptr;
  a->col_q = mx ? mx->col_q : nullptr;
  a->col_s = mx ? mx->col_s : nullptr;
  a->mx_cols = cols;
  a->mx_e5 = mx ? mx->e5m2 : 0;
  a->col_blocked = mx ? mx->col_blocked : 0;
  a->col_s_ld = a->col_blocked ? 4 * ((g->M_cap + 127) / 128 + g->E) : (g->M_cap + 31) / 32 + g->E;
}

// Persistent grid: one workgroup per usable CU (the kernel holds a CU's LDS),
// capped by an upper bound on the tile count (each expert adds at most one
// partial m-tile).
int persistent_grid(int cus, int cu_margin, int M_cap, int E, int ntiles_n) {
  int usable = cus - (cu_margin > 0 ? cu_margin : 0);
  if (usable < 1) usable = 1;
  long long bound = ((long long)(M_cap + GM_BM - 1) / GM_BM + E) * ntiles_n;
  if (bound < 1) bound = 1;
  return (int)(bound < usable ? bound : usable);
}

}  // namespace

namespace moe {

moe_status_t launch_activation_kernel(int kind, const GemmArgs& a, int grid, hipStream_t s) {
  const bool bwd = kind >= KIND_DGLU_PACKED;
  switch (a.ep.act) {
    case ACT_SWIGLU: return bwd ? launch_act_bwd_0(kind, a, grid, s) : launch_act_fwd_0(kind, a, grid, s);
    case ACT_GEGLU: return bwd ? launch_act_bwd_1(kind, a, grid, s) : launch_act_fwd_1(kind, a, grid, s);
    case ACT_GEGLU_TANH:
      return bwd ? launch_act_bwd_2(kind, a, grid, s) : launch_act_fwd_2(kind, a, grid, s);
    case ACT_SRELU: return bwd ? launch_act_bwd_3(kind, a, grid, s) : launch_act_fwd_3(kind, a, grid, s);
    default: return MOE_ERR_UNSUPPORTED;
  }
}

}  // namespace moe

extern "C" {

moe_status_t moe_init(int device) {
  if (device < 0 || device >= kMaxDevices) return MOE_ERR_DEVICE;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, device) != hipSuccess) return MOE_ERR_DEVICE;
  if (strncmp(prop.gcnArchName, "gfx950", 6) != 0) return MOE_ERR_DEVICE;
  g_num_cus[device] = prop.multiProcessorCount;
  return MOE_OK;
}

const char* moe_status_string(moe_status_t s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_NULL: return "a required pointer is NULL";
    case MOE_ERR_SHAPE: return "a size is out of range or not a supported multiple";
    case MOE_ERR_ALIGN: return "a pointer is not suitably aligned";
    case MOE_ERR_UNSUPPORTED: return "unsupported option combination";
    case MOE_ERR_LAUNCH: return "kernel launch failed";
    case MOE_ERR_DEVICE: return "no usable gfx950 device";
  }
  return "unknown status";
}

size_t moe_packed_weight_bytes(int E, int N, int K) {
  if (E <= 0 || N <= 0 || K <= 0) return 0;
  return (size_t)E * (size_t)((N + 255) / 256) * 256 * (size_t)K * 2;
}

size_t moe_packed_w1_bytes(int E, int H, int I) {
  if (I <= 0) return 0;
  return moe_packed_weight_bytes(E, 2 * I, H);
}

static moe_status_t launch_pack(const void* src, void* dst, int E, int N, int K, int mode, int I,
                                void* stream) {
  int cus;
  moe_status_t st = ensure_init(&cus);
  if (st != MOE_OK) return st;
  dim3 grid(K / 64, (N + 255) / 256, E);
  hipLaunchKernelGGL(pack_kernel, grid, dim3(256), 0, (hipStream_t)stream,
                     static_cast<const uint16_t*>(src), static_cast<uint16_t*>(dst), N, K, mode, I);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

moe_status_t moe_pack_weight(const void* src, int E, int N, int K, int src_layout, void* dst,
                             void* stream) {
  if (!src || !dst) return MOE_ERR_NULL;
  if (E < 1 || N < 64 || N % 64 != 0 || K < 64 || K % 64 != 0) return MOE_ERR_SHAPE;
  if (src_layout != MOE_B_NK && src_layout != MOE_B_KN) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(src) || !aligned16(dst)) return MOE_ERR_ALIGN;
  return launch_pack(src, dst, E, N, K, src_layout == MOE_B_NK ? PACK_NK : PACK_KN, 0, stream);
}

size_t moe_packed_mx_weight_bytes(int E, int N, int K) {
  if (E <= 0 || N <= 0 || K <= 0) return 0;
  return (size_t)E * (size_t)((N + 255) / 256) * 256 * (size_t)K;
}

size_t moe_packed_mx_scale_bytes(int E, int N, int K) {
  return moe_packed_mx_weight_bytes(E, N, K) / 32;
}

moe_status_t moe_pack_weight_mx(const void* src, int E, int N, int K, int src_layout, void* dst_q,
                                void* dst_s, void* stream) {
  if (!src || !dst_q || !dst_s) return MOE_ERR_NULL;
  if (E < 1 || N < 64 || N % 64 != 0 || K < 128 || K % 128 != 0) return MOE_ERR_SHAPE;
  if (src_layout != MOE_B_NK && src_layout != MOE_B_KN) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(src) || !aligned16(dst_q) || !aligned16(dst_s)) return MOE_ERR_ALIGN;
  int cus;
  moe_status_t st = ensure_init(&cus);
  if (st != MOE_OK) return st;
  dim3 grid(K / 128, (N + 255) / 256, E);
  hipLaunchKernelGGL(pack_mx_kernel, grid, dim3(256), 0, (hipStream_t)stream,
                     static_cast<const uint16_t*>(src), static_cast<uint8_t*>(dst_q),
                     static_cast<uint8_t*>(dst_s), N, K, src_layout == MOE_B_KN ? 1 : 0, 0);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

moe_status_t moe_repack_gate_up_mx(const void* w1, int E, int H, int I, void* dst_q, void* dst_s,
                                   void* stream) {
  if (!w1 || !dst_q || !dst_s) return MOE_ERR_NULL;
  if (E < 1 || H < 128 || H % 128 != 0 || I < 64 || I % 64 != 0) return MOE_ERR_SHAPE;
  if (!aligned16(w1) || !aligned16(dst_q) || !aligned16(dst_s)) return MOE_ERR_ALIGN;
  int cus;
  moe_status_t st = ensure_init(&cus);
  if (st != MOE_OK) return st;
  dim3 grid(H / 128, (2 * I + 255) / 256, E);
  hipLaunchKernelGGL(pack_mx_kernel, grid, dim3(256), 0, (hipStream_t)stream,
                     static_cast<const uint16_t*>(w1), static_cast<uint8_t*>(dst_q),
                     static_cast<uint8_t*>(dst_s), 2 * I, H, 1, I);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

moe_status_t moe_repack_gate_up(const void* w1, int E, int H, int I, void* w1_packed,
                                void* stream) {
  if (!w1 || !w1_packed) return MOE_ERR_NULL;
  if (E < 1 || H < 64 || H % 64 != 0 || I < 64 || I % 64 != 0) return MOE_ERR_SHAPE;
  if (!aligned16(w1) || !aligned16(w1_packed)) return MOE_ERR_ALIGN;
  return launch_pack(w1, w1_packed, E, 2 * I, H, PACK_GATEUP, I, stream);
}

moe_status_t moe_unpack_gate_up(const void* w1_packed, int E, int H, int I, void* w1,
                                void* stream) {
  if (!w1 || !w1_packed) return MOE_ERR_NULL;
  if (E < 1 || H < 64 || H % 64 != 0 || I < 64 || I % 64 != 0) return MOE_ERR_SHAPE;
  if (!aligned16(w1) || !aligned16(w1_packed)) return MOE_ERR_ALIGN;
  return launch_pack(w1_packed, w1, E, 2 * I, H, UNPACK_GATEUP, I, stream);
}

moe_status_t moe_route_group(const float* logits, const int32_t* topk_ids, int T, int E, int k,
                             int32_t* topk_ids_out, int32_t* counts, int32_t* offsets,
                             int32_t* dst, int32_t* src, const void* x, int H, void* xg,
                             void* stream) {
  if ((logits == nullptr) == (topk_ids == nullptr)) return MOE_ERR_NULL;
  if (!topk_ids_out || !counts || !offsets || !dst || !src) return MOE_ERR_NULL;
  if ((x == nullptr) != (xg == nullptr)) return MOE_ERR_NULL;
  if (T < 0 || E < 1 || E > kMaxExperts || k < 1 || k > 16 || k > E) return MOE_ERR_SHAPE;
  if ((long long)T * k >= (1LL << 31)) return MOE_ERR_SHAPE;
  if (x && (H < 8 || H % 8 != 0)) return MOE_ERR_SHAPE;
  if (x && (!aligned16(x) || !aligned16(xg))) return MOE_ERR_ALIGN;
  int cus;
  moe_status_t st = ensure_init(&cus);
  if (st != MOE_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  const int TK = T * k;
  if (logits) {
    if (T > 0) {
      // one token per 16, 32 or 64 lanes
      const int L = E <= 16 ? 16 : (E <= 32 ? 32 : 64);
      const int per_block = 4 * (64 / L);
      const dim3 grid((T + per_block - 1) / per_block);
      if (L == 16)
        hipLaunchKernelGGL(topk_kernel<16>, grid, dim3(256), 0, s, logits, T, E, k, topk_ids_out);
      else if (L == 32)
        hipLaunchKernelGGL(topk_kernel<32>, grid, dim3(256), 0, s, logits, T, E, k, topk_ids_out);
      else
        hipLaunchKernelGGL(topk_kernel<64>, grid, dim3(256), 0, s, logits, T, E, k, topk_ids_out);
    }
  } else if (topk_ids != topk_ids_out && TK > 0) {
    if (hipMemcpyAsync(topk_ids_out, topk_ids, (size_t)TK * 4, hipMemcpyDeviceToDevice, s) !=
        hipSuccess)
      return MOE_ERR_LAUNCH;
  }
  // chunks of C pairs (C >= 2E, so that the per-chunk counts fit in src; see
  // group_count_kernel)
  int C = 1024;
  while (C < 2 * E) C *= 2;
  const int nchunks = (TK + C - 1) / C;
  if (nchunks > 1) {
    hipLaunchKernelGGL(group_count_kernel, dim3(nchunks), dim3(256), 0, s, topk_ids_out, TK, E, C, src);
    hipLaunchKernelGGL(group_scan_kernel, dim3(1), dim3(1024), 0, s, nchunks, E, src, counts, offsets);
  }
  // (with no pairs the single rank workgroup still writes zero counts)
  hipLaunchKernelGGL(group_rank_kernel, dim3(nchunks > 1 ? nchunks : 1), dim3(256), 0, s,
                     topk_ids_out, TK, E, C, nchunks > 1 ? src : nullptr, dst, counts, offsets);
  if (TK > 0) {
    const int grid = min((TK + 3) / 4, cus * 32);   // 4 pairs (one per wave) per workgroup step
    hipLaunchKernelGGL(group_scatter_kernel, dim3(grid), dim3(256), 0, s, topk_ids_out, TK, k, E, dst,
                       offsets, src, static_cast<const uint16_t*>(x), H, static_cast<uint16_t*>(xg));
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

moe_status_t moe_group_gemm_glu_fwd(const void* xg, const moe_groups_t* groups,
                                    const void* w1_packed, int H, int I,
                                    const moe_epilogue_t* ep, void* y, void* preact,
                                    const moe_mx_out_t* mx, int cu_margin, void* stream) {
  moe_status_t st = check_groups(groups);
  if (st != MOE_OK) return st;
  if (!xg || !w1_packed || !ep) return MOE_ERR_NULL;
  if ((st = check_mx(mx)) != MOE_OK) return st;
  if (H < 64 || H % 64 != 0 || I < 64 || I % 64 != 0) return MOE_ERR_SHAPE;
  if (ep->gated != 0 && ep->gated != 1) return MOE_ERR_UNSUPPORTED;
  const bool gated = ep->gated == 1;
  if (!aligned16(xg) || !aligned16(w1_packed) || (y && !aligned16(y)) ||
      (preact && !aligned16(preact)))
    return MOE_ERR_ALIGN;
  GemmArgs a;
  memset(&a, 0, sizeof(a));
  if ((st = fill_epilogue(ep, &a.ep)) != MOE_OK) return st;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  fill_groups(&a, groups);
  a.A = static_cast<const uint16_t*>(xg);
  a.B = static_cast<const uint16_t*>(w1_packed);
  // gated: the gate/up-repacked W1 (N = 2I packed columns); non-gated: W1
  // [E][H][I] packed by moe_pack_weight (N = I plain columns)
  a.b_estride = gated ? (long long)moe_packed_w1_bytes(1, H, I) / 2
                      : (long long)moe_packed_weight_bytes(1, I, H) / 2;
  a.ldb = H;
  a.N = gated ? 2 * I : I;
  a.K = H;
  a.I = I;
  a.C = static_cast<uint16_t*>(y);
  a.preact = static_cast<uint16_t*>(preact);
  fill_mx(&a, mx, I, groups);
  a.ntiles_n = (a.N + GM_BN - 1) / GM_BN;
  int grid = persistent_grid(cus, cu_margin, groups->M_cap, groups->E, a.ntiles_n);
  const int kind = !gated ? KIND_ACT : (a.row_q || a.col_q) ? KIND_GLU_MXO : KIND_GLU;
  return launch_activation_kernel(kind, a, grid, (hipStream_t)stream);
}

moe_status_t moe_group_gemm_glu_fwd_mx(const moe_operand_t* xg, const moe_groups_t* groups,
                                       const moe_operand_t* w1, int H, int I,
                                       const moe_epilogue_t* ep, void* y, void* preact,
                                       const moe_mx_out_t* mx, int cu_margin, void* stream) {
  moe_status_t st = check_groups(groups);
  if (st != MOE_OK) return st;
  if (!xg || !w1 || !ep || !xg->data || !xg->scales || !w1->data || !w1->scales) return MOE_ERR_NULL;
  if ((st = check_mx(mx)) != MOE_OK) return st;
  if (H < 128 || H % 128 != 0 || I < 64 || I % 64 != 0) return MOE_ERR_SHAPE;
  if (ep->gated != 1 || xg->dtype != MOE_DT_MXFP8 || w1->dtype != MOE_DT_MXFP8 ||
      w1->layout != MOE_B_PACKED)
    return MOE_ERR_UNSUPPORTED;
  if (!aligned16(xg->data) || !aligned16(xg->scales) || !aligned16(w1->data) ||
      !aligned16(w1->scales) || (y && !aligned16(y)) || (preact && !aligned16(preact)))
    return MOE_ERR_ALIGN;
  GemmArgs a;
  memset(&a, 0, sizeof(a));
  if ((st = fill_epilogue(ep, &a.ep)) != MOE_OK) return st;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  fill_groups(&a, groups);
  a.A = static_cast<const uint16_t*>(xg->data);
  a.a_scales = xg->scales;
  a.B = static_cast<const uint16_t*>(w1->data);
  a.b_scales = w1->scales;
  a.b_estride = (long long)moe_packed_mx_weight_bytes(1, 2 * I, H);   // bytes = elements
  a.ldb = H;
  a.N = 2 * I;
  a.K = H;
  a.I = I;
  a.C = static_cast<uint16_t*>(y);
  a.preact = static_cast<uint16_t*>(preact);
  fill_mx(&a, mx, I, groups);
  a.ntiles_n = (2 * I + GM_BN - 1) / GM_BN;
  int grid = persistent_grid(cus, cu_margin, groups->M_cap, groups->E, a.ntiles_n);
  return launch_activation_kernel((a.row_q || a.col_q) ? KIND_MXIN_GLU_MXO : KIND_MXIN_GLU, a,
                                  grid, (hipStream_t)stream);
}

moe_status_t moe_group_gemm_dglu_bwd(const void* dy2, const moe_operand_t* w2, int H, int I,
                                     const moe_groups_t* groups, const void* preact,
                                     const moe_epilogue_t* ep, void* dgu,
                                     const moe_mx_out_t* mx, int cu_margin, void* stream) {
  moe_status_t st = check_groups(groups);
  if (st != MOE_OK) return st;
  if (!dy2 || !w2 || !w2->data || !preact || !ep) return MOE_ERR_NULL;
  if ((st = check_mx(mx)) != MOE_OK) return st;
  if (H < 64 || H % 64 != 0 || I < 64 || I % 64 != 0) return MOE_ERR_SHAPE;
  if ((ep->gated != 0 && ep->gated != 1) || w2->dtype != MOE_DT_BF16) return MOE_ERR_UNSUPPORTED;
  const bool gated = ep->gated == 1;
  if (!gated && (ep->dbias_out || ep->drow_scale_out)) return MOE_ERR_UNSUPPORTED;
  if (w2->layout != MOE_B_NK && w2->layout != MOE_B_PACKED) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(dy2) || !aligned16(w2->data) || !aligned16(preact) || (dgu && !aligned16(dgu)))
    return MOE_ERR_ALIGN;
  GemmArgs a;
  memset(&a, 0, sizeof(a));
  if ((st = fill_epilogue(ep, &a.ep)) != MOE_OK) return st;
  a.ep.bias = nullptr;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  fill_groups(&a, groups);
  a.A = static_cast<const uint16_t*>(dy2);
  a.B = static_cast<const uint16_t*>(w2->data);  // W2_e [I][H] = W2_e^T stored [N=I][K=H]
  const bool w2_packed = w2->layout == MOE_B_PACKED;
  a.b_estride = w2_packed ? (long long)moe_packed_weight_bytes(1, I, H) / 2 : (long long)I * H;
  a.ldb = H;
  a.N = I;
  a.K = H;
  a.I = I;
  a.C = static_cast<uint16_t*>(dgu);
  a.preact = const_cast<uint16_t*>(static_cast<const uint16_t*>(preact));
  fill_mx(&a, mx, gated ? 2 * I : I, groups);
  a.ntiles_n = (I + GM_BN - 1) / GM_BN;
  int grid = persistent_grid(cus, cu_margin, groups->M_cap, groups->E, a.ntiles_n);
  const bool grads = a.ep.dbias_out || a.ep.drs_out;
  const int kind = !gated ? (w2_packed ? KIND_DACT_PACKED : KIND_DACT_NK)
                   : grads ? (w2_packed ? KIND_DGLU_G_PACKED : KIND_DGLU_G_NK)
                           : (w2_packed ? KIND_DGLU_PACKED : KIND_DGLU_NK);
  return launch_activation_kernel(kind, a, grid, (hipStream_t)stream);
}

static moe_status_t group_gemm_mxfp4(const moe_operand_t* a_op, const moe_operand_t* b_op, int N, int K,
                                     const moe_groups_t* groups, void* c_bf16, const moe_mx_out_t* mx,
                                     int cu_margin, hipStream_t stream) {
  const bool a4 = a_op->dtype == MOE_DT_MXFP4;
  if ((!a4 && a_op->dtype != MOE_DT_MXFP8) || b_op->layout != MOE_B_NK) return MOE_ERR_UNSUPPORTED;
  if (mx && (mx->row_q || mx->col_q)) return MOE_ERR_UNSUPPORTED;
  const bool rows = groups->M_cap > 0;   // without rows A and C may be NULL
  if (!b_op->scales || (rows && (!a_op->data || !a_op->scales || !c_bf16))) return MOE_ERR_NULL;
  if (K % 32 != 0 || K >= kMaxMx4K || N >= kMaxMx4N) return MOE_ERR_SHAPE;
  if (!aligned16(a_op->data) || !aligned16(b_op->data) || !aligned16(c_bf16)) return MOE_ERR_ALIGN;
  const int M = groups->M_cap, E = groups->E;
  const long long EN = (long long)E * N;
  if (overlap({{c_bf16, bytes_of(M, N)}, {groups->offsets_out, bytes_of(1, E + 1, 32)}, {groups->status_out, 4}},
              {{a_op->data, bytes_of(M, K, a4 ? 4 : 8)}, {a_op->scales, bytes_of(M, K / 32, 8)},
               {b_op->data, bytes_of(EN, K, 4)}, {b_op->scales, bytes_of(EN, K / 32, 8)},
               {groups->counts, bytes_of(1, E, 32)}}))
    return MOE_ERR_UNSUPPORTED;
  int cus;
  moe_status_t st = ensure_init(&cus);
  if (st != MOE_OK) return st;
  Mx4Args a;
  memset(&a, 0, sizeof(a));
  a.A = static_cast<const uint8_t*>(a_op->data);
  a.a_scales = a_op->scales;
  a.B = static_cast<const uint8_t*>(b_op->data);
  a.b_scales = b_op->scales;
  a.M_cap = groups->M_cap;
  a.N = N;
  a.K = K;
  a.counts = groups->counts;
  a.E = groups->E;
  a.offsets_out = groups->offsets_out;
  a.status_out = groups->status_out;
  a.C = static_cast<uint16_t*>(c_bf16);
  int usable = cus - (cu_margin > 0 ? cu_margin : 0);
  if (usable < 1) usable = 1;
  return launch_mx4_gemm(a, a4, usable, stream);
}

moe_status_t moe_group_gemm_quant(const moe_operand_t* a_op, const moe_operand_t* b_op, int N,
                                  int K, const moe_groups_t* groups, void* c_bf16,
                                  const moe_mx_out_t* mx, int cu_margin, void* stream) {
  moe_status_t st = check_groups(groups);
  if (st != MOE_OK) return st;
  if (!a_op || !b_op || !b_op->data) return MOE_ERR_NULL;
  if (!a_op->data && (b_op->dtype != MOE_DT_MXFP4 || groups->M_cap > 0)) return MOE_ERR_NULL;
  if ((st = check_mx(mx)) != MOE_OK) return st;
  if (N < 64 || N % 64 != 0 || K < 32) return MOE_ERR_SHAPE;
  if (b_op->dtype == MOE_DT_MXFP4)   // MXFP4 weights (K % 32 == 0, checked there)
    return group_gemm_mxfp4(a_op, b_op, N, K, groups, c_bf16, mx, cu_margin, (hipStream_t)stream);
  if (K < 64 || K % 64 != 0) return MOE_ERR_SHAPE;
  const bool a_e5 = a_op->dtype == MOE_DT_MXFP8_E5M2;
  const bool mx_in = a_op->dtype == MOE_DT_MXFP8 || a_e5 || b_op->dtype != MOE_DT_BF16;
  if (mx_in) {   // MXFP8 (A e4m3 or e5m2) x MXFP8 e4m3 only, weight from moe_pack_weight_mx
    if ((a_op->dtype != MOE_DT_MXFP8 && !a_e5) || b_op->dtype != MOE_DT_MXFP8 ||
        b_op->layout != MOE_B_PACKED)
      return MOE_ERR_UNSUPPORTED;
    if (!a_op->scales || !b_op->scales) return MOE_ERR_NULL;
    if (K % 128 != 0) return MOE_ERR_SHAPE;
    if (!aligned16(a_op->scales) || !aligned16(b_op->scales)) return MOE_ERR_ALIGN;
  } else if (a_op->dtype != MOE_DT_BF16 || b_op->dtype != MOE_DT_BF16) {
    return MOE_ERR_UNSUPPORTED;
  }
  if (!aligned16(a_op->data) || !aligned16(b_op->data) || (c_bf16 && !aligned16(c_bf16)))
    return MOE_ERR_ALIGN;
  GemmArgs a;
  memset(&a, 0, sizeof(a));
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  fill_groups(&a, groups);
  a.A = static_cast<const uint16_t*>(a_op->data);
  a.B = static_cast<const uint16_t*>(b_op->data);
  a.N = N;
  a.K = K;
  a.C = static_cast<uint16_t*>(c_bf16);
  fill_mx(&a, mx, N, groups);
  a.ntiles_n = (N + GM_BN - 1) / GM_BN;
  if (mx_in) {
    a.a_scales = static_cast<const uint8_t*>(a_op->scales);
    a.b_scales = static_cast<const uint8_t*>(b_op->scales);
    a.ldb = K;
    a.b_estride = (long long)moe_packed_mx_weight_bytes(1, N, K);   // bytes = elements
    int grid = persistent_grid(cus, cu_margin, groups->M_cap, groups->E, a.ntiles_n);
    return launch_group_gemm_mx(a, a_e5, grid, (hipStream_t)stream);
  }
  int blay;
  switch (b_op->layout) {
    case MOE_B_KN: blay = BL_KN; a.ldb = N; a.b_estride = (long long)K * N; break;
    case MOE_B_NK: blay = BL_NK; a.ldb = K; a.b_estride = (long long)N * K; break;
    case MOE_B_PACKED:
      blay = BL_PACKED; a.ldb = K; a.b_estride = (long long)moe_packed_weight_bytes(1, N, K) / 2;
      break;
    default: return MOE_ERR_UNSUPPORTED;
  }
  int grid = persistent_grid(cus, cu_margin, groups->M_cap, groups->E, a.ntiles_n);
  if (blay == BL_PACKED) return launch_group_gemm_bwd(EPI_STORE, blay, a, grid, (hipStream_t)stream);
  return launch_group_gemm_fwd(EPI_STORE, blay, a, grid, (hipStream_t)stream);
}

moe_status_t moe_group_gemm_wgrad(const void* a, const void* b, int P, int Q,
                                  const moe_groups_t* groups, float* c, int accumulate,
                                  int cu_margin, void* stream) {
  moe_status_t st = check_groups(groups);
  if (st != MOE_OK) return st;
  if (!a || !b || !c) return MOE_ERR_NULL;
  if (P < 64 || P % 64 != 0 || Q < 64 || Q % 64 != 0) return MOE_ERR_SHAPE;
  if (!aligned16(a) || !aligned16(b) || !aligned16(c)) return MOE_ERR_ALIGN;
  GemmArgs g;
  memset(&g, 0, sizeof(g));
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  fill_groups(&g, groups);
  g.A = static_cast<const uint16_t*>(a);
  g.B = static_cast<const uint16_t*>(b);
  g.ldb = Q;
  g.N = Q;
  g.K = 64;                       // unused: each tile reduces over its group's rows
  g.wg_P = P;
  g.ntiles_m = (P + GM_BM - 1) / GM_BM;
  g.ntiles_n = (Q + GM_BN - 1) / GM_BN;
  g.Cf = c;
  g.accumulate = accumulate ? 1 : 0;
  int usable = cus - (cu_margin > 0 ? cu_margin : 0);
  if (usable < 1) usable = 1;
  const long long tiles = (long long)groups->E * g.ntiles_m * g.ntiles_n;
  const int grid = (int)(tiles < usable ? tiles : usable);
  return launch_group_gemm_wgrad(g, grid, (hipStream_t)stream);
}

moe_status_t moe_group_gemm_wgrad_mx(const moe_operand_t* a, const moe_operand_t* b, int P, int Q,
                                     const moe_groups_t* groups, float* c, int accumulate,
                                     int cu_margin, void* stream) {
  moe_status_t st = check_groups(groups);
  if (st != MOE_OK) return st;
  if (!a || !b || !c || !a->data || !b->data || !a->scales || !b->scales) return MOE_ERR_NULL;
  auto is_mx = [](int dt) { return dt == MOE_DT_MXFP8 || dt == MOE_DT_MXFP8_E5M2; };
  if (!is_mx(a->dtype) || !is_mx(b->dtype)) return MOE_ERR_UNSUPPORTED;
  if (P < 64 || P % 64 != 0 || Q < 64 || Q % 64 != 0) return MOE_ERR_SHAPE;
  if (!aligned16(a->data) || !aligned16(b->data) || !aligned4(a->scales) || !aligned4(b->scales) ||
      !aligned16(c))
    return MOE_ERR_ALIGN;
  const int S = 4 * ((groups->M_cap + 127) / 128 + groups->E);   // slots per copied column
  GemmArgs g;
  memset(&g, 0, sizeof(g));
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  fill_groups(&g, groups);
  g.A = static_cast<const uint16_t*>(a->data);
  g.B = static_cast<const uint16_t*>(b->data);
  g.a_scales = a->scales;
  g.b_scales = b->scales;
  g.K = 32 * S;                   // bytes per copied column (row of each operand)
  g.ldb = 32 * S;
  g.N = Q;
  g.wg_P = P;
  g.ntiles_m = (P + GM_BM - 1) / GM_BM;
  g.ntiles_n = (Q + GM_BN - 1) / GM_BN;
  g.Cf = c;
  g.accumulate = accumulate ? 1 : 0;
  int usable = cus - (cu_margin > 0 ? cu_margin : 0);
  if (usable < 1) usable = 1;
  const long long tiles = (long long)groups->E * g.ntiles_m * g.ntiles_n;
  const int grid = (int)(tiles < usable ? tiles : usable);
  return launch_group_gemm_wgrad_mx(g, a->dtype == MOE_DT_MXFP8_E5M2, b->dtype == MOE_DT_MXFP8_E5M2,
                                    grid, (hipStream_t)stream);
}

moe_status_t moe_glu_unfused(const void* z, const moe_groups_t* groups, int I,
                             const moe_epilogue_t* ep, void* y, void* stream) {
  moe_status_t st = check_groups(groups);
  if (st != MOE_OK) return st;
  if (!z || !y || !ep) return MOE_ERR_NULL;
  if (I < 64 || I % 64 != 0) return MOE_ERR_SHAPE;
  if (ep->gated != 1) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(z) || !aligned16(y)) return MOE_ERR_ALIGN;
  EpiParams e;
  if ((st = fill_epilogue(ep, &e)) != MOE_OK) return st;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  hipLaunchKernelGGL(glu_unfused_kernel, dim3(cus * 8), dim3(256), 0, (hipStream_t)stream,
                     static_cast<const uint16_t*>(z), groups->counts, groups->E, groups->M_cap, I,
                     e, static_cast<uint16_t*>(y));
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

moe_status_t moe_dglu_unfused(const void* g, const void* z, const moe_groups_t* groups, int I,
                              const moe_epilogue_t* ep, void* dgu, void* stream) {
  moe_status_t st = check_groups(groups);
  if (st != MOE_OK) return st;
  if (!g || !z || !dgu || !ep) return MOE_ERR_NULL;
  if (I < 64 || I % 64 != 0) return MOE_ERR_SHAPE;
  if (ep->gated != 1) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(g) || !aligned16(z) || !aligned16(dgu)) return MOE_ERR_ALIGN;
  EpiParams e;
  if ((st = fill_epilogue(ep, &e)) != MOE_OK) return st;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  hipLaunchKernelGGL(dglu_unfused_kernel, dim3(cus * 8), dim3(256), 0, (hipStream_t)stream,
                     static_cast<const uint16_t*>(g), static_cast<const uint16_t*>(z), groups->counts,
                     groups->E, groups->M_cap, I, e, static_cast<uint16_t*>(dgu));
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

moe_status_t moe_mxfp8_quantize(const void* v, int R, int C, const moe_groups_t* groups,
                                const moe_mx_out_t* mx, void* stream) {
  if (!v || !mx) return MOE_ERR_NULL;
  moe_status_t st = check_mx(mx);
  if (st != MOE_OK) return st;
  if (groups && (st = check_groups(groups)) != MOE_OK) return st;
  if (groups && groups->M_cap != R) return MOE_ERR_SHAPE;
  if (R < 0 || C < 32 || C % 32 != 0) return MOE_ERR_SHAPE;
  if (!aligned16(v)) return MOE_ERR_ALIGN;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  const int* counts = groups ? groups->counts : nullptr;
  const int E = groups ? groups->E : 0;
  if (mx->row_q && R > 0) {
    hipLaunchKernelGGL(mx_rows_kernel, dim3(cus * 8), dim3(256), 0, s,
                       static_cast<const uint16_t*>(v), R, C, counts, E, mx->row_q, mx->row_s,
                       mx->e5m2);
  }
  if (mx->col_q && R > 0) {
    const int Eg = groups ? E : 0;
    int s_ld = mx->col_blocked ? 4 * ((R + 127) / 128 + Eg) : (R + 31) / 32 + Eg;
    if (mx->col_blocked) {   // LDS-staged, 256 rows x 64 columns per item
      const long long items = (long long)((R + 255) / 256 + Eg) * ((C + 63) / 64);
      const int grid = (int)(items < (long long)cus * 6 ? items : (long long)cus * 6);
      hipLaunchKernelGGL(mx_cols_ktiled_kernel, dim3(grid), dim3(256), 0, s,
                         static_cast<const uint16_t*>(v), R, C, counts, E, mx->col_q, mx->col_s, s_ld,
                         mx->e5m2);
    } else {
      long long by = s_ld;
      int gy = (int)(by < 65535 ? by : 65535);
      hipLaunchKernelGGL(mx_cols_kernel, dim3((C + 255) / 256, gy), dim3(256), 0, s,
                         static_cast<const uint16_t*>(v), R, C, counts, E, mx->col_q, mx->col_s, s_ld,
                         mx->e5m2, mx->col_blocked);
    }
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

static moe_status_t check_router(const void* logits, int logits_dtype, int T, int E, int k,
                                 const moe_router_t* r, RouterArgs* out) {
  if ((!logits && T != 0) || !r) return MOE_ERR_NULL;
  if (T < 0 || T > kMaxRouterTokens || E < 1 || E > kMaxExperts || k < 1 || k > kMaxTopk || k > E)
    return MOE_ERR_SHAPE;
  if (logits_dtype != MOE_DT_BF16 && logits_dtype != MOE_DT_FP32) return MOE_ERR_UNSUPPORTED;
  if ((r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) ||
      (r->group_score != MOE_GROUP_MAX && r->group_score != MOE_GROUP_TOP2) ||
      (r->renorm != 0 && r->renorm != 1))
    return MOE_ERR_UNSUPPORTED;
  if (r->n_groups < 1 || r->n_groups > kMaxRouterGroups || E % r->n_groups != 0 || r->topk_groups < 1 ||
      r->topk_groups > r->n_groups || k > r->topk_groups * (E / r->n_groups))
    return MOE_ERR_SHAPE;
  const bool top2 = r->n_groups > 1 && r->group_score == MOE_GROUP_TOP2;
  if ((top2 && E / r->n_groups < 2) || !isfinite(r->scale)) return MOE_ERR_SHAPE;
  if (!aligned16(logits) || (r->bias && !aligned4(r->bias))) return MOE_ERR_ALIGN;
  out->logits = logits;
  out->bias = r->bias;
  out->T = T;
  out->E = E;
  out->k = k;
  out->sigmoid = r->score == MOE_SCORE_SIGMOID;
  out->n_groups = r->n_groups;
  out->topk_groups = r->topk_groups;
  out->top2 = top2;
  out->renorm = r->renorm;
  out->scale = r->scale;
  return MOE_OK;
}

moe_status_t moe_router_topk(const void* logits, int logits_dtype, int T, int E, int k,
                             const moe_router_t* router, int32_t* ids, float* weights, void* stream) {
  RouterArgs a;
  moe_status_t st = check_router(logits, logits_dtype, T, E, k, router, &a);
  if (st != MOE_OK) return st;
  if (T != 0 && (!ids || !weights)) return MOE_ERR_NULL;
  if (!aligned4(ids) || !aligned4(weights)) return MOE_ERR_ALIGN;
  const size_t pairs = bytes_of(T, k, 32);
  if (overlap({{ids, pairs}, {weights, pairs}},
              {{logits, bytes_of(T, E, logits_dtype == MOE_DT_BF16 ? 16 : 32)}, {a.bias, bytes_of(1, E, 32)}}))
    return MOE_ERR_UNSUPPORTED;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  return launch_router(a, logits_dtype == MOE_DT_BF16, ids, weights, (hipStream_t)stream);
}

moe_status_t moe_router_topk_bwd(const void* logits, int logits_dtype, int T, int E, int k,
                                 const moe_router_t* router, const int32_t* ids, const float* dweights,
                                 void* dlogits, void* stream) {
  RouterArgs a;
  moe_status_t st = check_router(logits, logits_dtype, T, E, k, router, &a);
  if (st != MOE_OK) return st;
  if (T != 0 && (!ids || !dweights || !dlogits)) return MOE_ERR_NULL;
  if (!aligned4(ids) || !aligned4(dweights) || !aligned16(dlogits)) return MOE_ERR_ALIGN;
  const size_t pairs = bytes_of(T, k, 32), rows = bytes_of(T, E, logits_dtype == MOE_DT_BF16 ? 16 : 32);
  if (overlap({{dlogits, rows}}, {{logits, rows}, {ids, pairs}, {dweights, pairs}})) return MOE_ERR_UNSUPPORTED;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  return launch_router_bwd(a, logits_dtype == MOE_DT_BF16, ids, dweights, dlogits, (hipStream_t)stream);
}

static moe_status_t check_combine(int M_cap, int H, const int32_t* dst, int T, int k, const float* weights) {
  if (!dst && T != 0) return MOE_ERR_NULL;
  if (M_cap < 0 || T < 0 || k < 1 || k > kMaxTopk || H < 8 || H % 8 != 0 || H > kMaxCombineH)
    return MOE_ERR_SHAPE;
  if (!aligned4(dst) || (weights && !aligned4(weights))) return MOE_ERR_ALIGN;
  return MOE_OK;
}

moe_status_t moe_combine(const void* y, int M_cap, int H, const int32_t* dst, const float* weights, int T,
                         int k, const void* residual, void* out, void* stream) {
  moe_status_t st = check_combine(M_cap, H, dst, T, k, weights);
  if (st != MOE_OK) return st;
  if ((!y && M_cap != 0) || (!out && T != 0)) return MOE_ERR_NULL;
  if (!aligned16(y) || !aligned16(out) || (residual && !aligned16(residual))) return MOE_ERR_ALIGN;
  const size_t pairs = bytes_of(T, k, 32), rows = bytes_of(T, H);
  if (overlap({{out, rows}}, {{y, bytes_of(M_cap, H)}, {dst, pairs}, {weights, pairs},
                              {residual == out ? nullptr : residual, rows}}))
    return MOE_ERR_UNSUPPORTED;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  return launch_combine(static_cast<const uint16_t*>(y), M_cap, H, dst, weights, T, k,
                        static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(out),
                        (hipStream_t)stream);
}

moe_status_t moe_combine_bwd(const void* dout, const void* y, int M_cap, int H, const int32_t* dst,
                             const float* weights, int T, int k, void* dy, float* dweights, void* stream) {
  moe_status_t st = check_combine(M_cap, H, dst, T, k, weights);
  if (st != MOE_OK) return st;
  if ((!dout && T != 0) || (!dy && !dweights && M_cap != 0 && T != 0) || (dweights && !y && M_cap != 0))
    return MOE_ERR_NULL;
  if (!aligned16(dout) || (y && !aligned16(y)) || (dy && !aligned16(dy)) ||
      (dweights && !aligned4(dweights)))
    return MOE_ERR_ALIGN;
  const size_t pairs = bytes_of(T, k, 32), rows = bytes_of(M_cap, H);
  if (overlap({{dy, rows}, {dweights, pairs}},
              {{dout, bytes_of(T, H)}, {y, rows}, {dst, pairs}, {weights, pairs}}))
    return MOE_ERR_UNSUPPORTED;
  if (!dy && !dweights) return MOE_OK;   // no tokens or no rows
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  return launch_combine_bwd(static_cast<const uint16_t*>(dout), static_cast<const uint16_t*>(y), M_cap, H,
                            dst, weights, T, k, static_cast<uint16_t*>(dy), dweights, (hipStream_t)stream);
}

moe_status_t moe_add_rmsnorm(const void* x, const void* residual, const void* weight, int T, int H,
                             float eps, void* h, void* y, float* rstd, const moe_mx_out_t* mx, void* stream) {
  if ((!x && T != 0) || !weight) return MOE_ERR_NULL;
  moe_status_t st = check_mx(mx);
  if (st != MOE_OK) return st;
  if (mx && mx->col_q) return MOE_ERR_UNSUPPORTED;
  const bool q = mx && mx->row_q;
  if (!h && !y && !rstd && !q && T != 0) return MOE_ERR_NULL;
  if (T < 0 || H < 8 || H % 8 != 0 || H > kNormMaxH || (q && H % 32 != 0)) return MOE_ERR_SHAPE;
  if (!(eps >= 0.0f) || !isfinite(eps)) return MOE_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(weight) || (residual && !aligned16(residual)) || (h && !aligned16(h)) ||
      (y && !aligned16(y)) || (rstd && !aligned4(rstd)))
    return MOE_ERR_ALIGN;
  const size_t rows = bytes_of(T, H);
  if (overlap({{y, rows}, {rstd, bytes_of(T, 1, 32)}, {q ? mx->row_q : nullptr, rows / 2},
               {q ? mx->row_s : nullptr, rows / 64}, {h, rows}},
              {{x == h ? nullptr : x, rows}, {residual == h ? nullptr : residual, rows}, {weight, bytes_of(1, H)}}))
    return MOE_ERR_UNSUPPORTED;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.weight = static_cast<const uint16_t*>(weight);
  a.T = T;
  a.H = H;
  a.eps = eps;
  a.inv_h = 1.0 / H;
  a.h = static_cast<uint16_t*>(h);
  a.y = static_cast<uint16_t*>(y);
  a.rstd = rstd;
  a.q = q ? mx->row_q : nullptr;
  a.s = q ? mx->row_s : nullptr;
  a.e5 = q ? mx->e5m2 : 0;
  return launch_add_rmsnorm(a, (hipStream_t)stream);
}

size_t moe_add_rmsnorm_bwd_workspace_bytes(int T, int H) {
  if (T <= 0 || H <= 0) return 0;
  return (size_t)norm_bwd_parts(T) * (size_t)H * sizeof(float);
}

moe_status_t moe_add_rmsnorm_bwd(const void* dy, const void* h, const void* weight, const float* rstd,
                                 const void* dh, int T, int H, void* dx, float* dweight, int accumulate,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!weight || (T != 0 && (!dy || !h || !rstd || (!dx && !dweight)))) return MOE_ERR_NULL;
  if (T < 0 || H < 8 || H % 8 != 0 || H > kNormMaxH) return MOE_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_UNSUPPORTED;
  if (dweight && T > 0) {
    if (!workspace) return MOE_ERR_NULL;
    if (workspace_bytes < moe_add_rmsnorm_bwd_workspace_bytes(T, H)) return MOE_ERR_SHAPE;
  }
  if (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned4(rstd) || (dh && !aligned16(dh)) ||
      (dx && !aligned16(dx)) || (dweight && !aligned4(dweight)) || (workspace && !aligned16(workspace)))
    return MOE_ERR_ALIGN;
  const size_t rows = bytes_of(T, H);
  if (overlap({{dx, rows}, {dweight, bytes_of(1, H, 32)},
               {dweight ? workspace : nullptr, moe_add_rmsnorm_bwd_workspace_bytes(T, H)}},
              {{dy, rows}, {h, rows}, {weight, bytes_of(1, H)}, {rstd, bytes_of(T, 1, 32)},
               {dh == dx ? nullptr : dh, rows}}))
    return MOE_ERR_UNSUPPORTED;
  int cus;
  moe_status_t st = ensure_init(&cus);
  if (st != MOE_OK) return st;
  NormBwdArgs a;
  memset(&a, 0, sizeof(a));
  a.dy = static_cast<const uint16_t*>(dy);
  a.h = static_cast<const uint16_t*>(h);
  a.weight = static_cast<const uint16_t*>(weight);
  a.rstd = rstd;
  a.dh = static_cast<const uint16_t*>(dh);
  a.T = T;
  a.H = H;
  a.dx = static_cast<uint16_t*>(dx);
  a.part = dweight ? static_cast<float*>(workspace) : nullptr;
  return launch_add_rmsnorm_bwd(a, dweight, accumulate, (hipStream_t)stream);
}

moe_status_t moe_mxfp4_quantize(const void* v, int R, int C, const moe_groups_t* groups, uint8_t* q,
                                uint8_t* s, void* stream) {
  if (R != 0 && (!v || !q || !s)) return MOE_ERR_NULL;
  moe_status_t st;
  if (groups && (st = check_groups(groups)) != MOE_OK) return st;
  if (groups && groups->M_cap != R) return MOE_ERR_SHAPE;
  if (R < 0 || C < 32 || C % 32 != 0) return MOE_ERR_SHAPE;
  if (!aligned16(v) || !aligned16(q)) return MOE_ERR_ALIGN;
  if (overlap({{q, bytes_of(R, C, 4)}, {s, bytes_of(R, C / 32, 8)}},
              {{v, bytes_of(R, C)}, {groups ? groups->counts : nullptr, groups ? bytes_of(1, groups->E, 32) : 0}}))
    return MOE_ERR_UNSUPPORTED;
  int cus;
  if ((st = ensure_init(&cus)) != MOE_OK) return st;
  return launch_mx4_rows(static_cast<const uint16_t*>(v), R, C, groups ? groups->counts : nullptr,
                         groups ? groups->E : 0, q, s, cus, (hipStream_t)stream);
}

moe_status_t moe_pack_weight_mxfp4(const void* src, int E, int N, int K, int src_layout, void* dst_q,
                                   void* dst_s, void* stream) {
  if (!src || !dst_q || !dst_s) return MOE_ERR_NULL;
  if (E < 1 || E > 65535 || N < 64 || N % 64 != 0 || K < 32 || K % 32 != 0 || K / 32 > 65535)
    return MOE_ERR_SHAPE;
  if ((long long)E * N >= (1LL << 31)) return MOE_ERR_SHAPE;
  if (src_layout != MOE_B_NK && src_layout != MOE_B_KN) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(src) || !aligned16(dst_q)) return MOE_ERR_ALIGN;
  const long long rows = (long long)E * N;
  if (overlap({{dst_q, bytes_of(rows, K, 4)}, {dst_s, bytes_of(rows, K / 32, 8)}}, {{src, bytes_of(rows, K)}}))
    return MOE_ERR_UNSUPPORTED;
  int cus;
  moe_status_t st = ensure_init(&cus);
  if (st != MOE_OK) return st;
  const uint16_t* w = static_cast<const uint16_t*>(src);
  uint8_t* q = static_cast<uint8_t*>(dst_q);
  uint8_t* sc = static_cast<uint8_t*>(dst_s);
  if (src_layout == MOE_B_NK)
    return launch_mx4_rows(w, E * N, K, nullptr, 0, q, sc, cus, (hipStream_t)stream);
  return launch_mx4_weight_kn(w, E, N, K, q, sc, (hipStream_t)stream);
}

}  // extern "C"
