/*
 * moe_glu.h -- C ABI of the sync-free MoE expert-MLP library for AMD MI355X
 * (CDNA4, gfx950): grouped GEMM over per-expert token groups whose sizes live
 * only in device memory, with the GLU activation, its backward and an MXFP8
 * quantize/transpose fused into the GEMM epilogues.
 *
 * Sources ("the pages"):
 *   [BLOG] "Boosting MoE Training Throughput with Advanced Fusion Kernels"
 *          (Spanish translation).  Its kernel family: GroupGemm + Quantize,
 *          GroupGemm + Activation + Quantize/Transpose, GroupGemm +
 *          dActivation + Quantize/Transpose; activations SwiGLU, GeGLU,
 *          sReLU with clamping and scaling.
 *   [MEGA] DeepSeek MegaMoE / DeepGEMM walkthrough (hnwysp.cn), §2.1 routing,
 *          §4.3 grouped GEMM over contiguous per-expert rows, §5.3 tail tiles.
 *
 * Conventions shared by every call:
 *   - Pointers are DEVICE pointers unless marked (host).  bf16 tensors are
 *     passed as 16-bit storage, e4m3fn elements and E8M0 scales as bytes.
 *     Every device pointer must be 16-byte aligned, except the MX outputs.
 *   - Every call is asynchronous on `stream` (a hipStream_t; NULL = the null
 *     stream).  No call allocates, synchronises, or reads device data back to
 *     the host, so each is legal inside hipStreamBeginCapture.
 *   - The caller owns every buffer.  The library keeps no per-call state.
 *   - Errors a host can see (null required pointer, bad shape, misalignment,
 *     unsupported option) return a nonzero status BEFORE anything launches.
 *     A failed launch returns MOE_ERR_LAUNCH.  Errors only the device can see
 *     (a negative count, counts summing past M_cap) set bits in
 *     groups->status_out and the work is clamped to M_cap rows; nothing is
 *     read or written out of bounds and no kernel traps.
 *   - Grouped rows: expert e owns rows [o_e, o_e + m_e) of every [M_cap][*]
 *     operand, o_e = sum_{j<e} m_j ([MEGA] §4.3).  Rows >= sum m_e, and all
 *     rows of a zero-row expert, are never written.
 *   - Calls on different streams are independent and re-entrant.
 */
#ifndef MOE_GLU_H
#define MOE_GLU_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_NULL = 1,         /* a required pointer is NULL */
  MOE_ERR_SHAPE = 2,        /* a size is out of range or not a supported multiple */
  MOE_ERR_ALIGN = 3,        /* a pointer is not 16-byte aligned */
  MOE_ERR_UNSUPPORTED = 4,  /* an option combination the library does not implement */
  MOE_ERR_LAUNCH = 5,       /* the HIP runtime rejected a launch */
  MOE_ERR_DEVICE = 6        /* no usable gfx950 device */
} moe_status_t;

typedef enum {
  MOE_ACT_SWIGLU = 0,       /* a(g) = g * sigmoid(alpha * g) */
  MOE_ACT_GEGLU = 1,        /* a(g) = g * Phi(g), exact erf form */
  MOE_ACT_GEGLU_TANH = 2,   /* a(g) = tanh approximation of g * Phi(g) */
  MOE_ACT_SRELU = 3         /* a(g) = max(g, 0)^2 */
} moe_act_t;

/* GLU epilogue ([BLOG] "Optimizando GLU vía epílogos GEMM fusionados": the
 * GLU splits FC1's output into an input (up) half and a gate half; the fused
 * epilogue also does feature scaling, clamping and bias addition).
 * With z = FC1 output + bias, g = z[:, :I] (gate), u = z[:, I:] (up):
 *     y = a(clamp(g, gate_lo, gate_hi)) * (clamp(u, up_lo, up_hi) + up_offset)
 *         * row_scale[row]
 * rounded to bf16 (round-to-nearest-even).  (host struct) */
typedef struct {
  int32_t act;              /* moe_act_t */
  int32_t gated;            /* 1: the gated (GLU) form y = a(g_c) * u_c; 0: the non-gated form
                               y = a(z) over I columns (no clamps, no up_offset; sReLU's
                               plain form), see moe_group_gemm_glu_fwd */
  float alpha;              /* SwiGLU gate scale inside the sigmoid; 1 = plain SiLU */
  float gate_lo, gate_hi;   /* clamp bounds on g; -inf/+inf = off */
  float up_lo, up_hi;       /* clamp bounds on u; -inf/+inf = off */
  float up_offset;          /* added to the clamped up value; 0 = off */
  const void* bias;         /* nullable: bf16 [E][2I] in PLAIN order (gate | up); [E][I] when
                               non-gated */
  const float* row_scale;   /* nullable: fp32 [M_cap], multiplies y per row */
  /* Per-tensor amax for an NVFP4-style recipe ([BLOG] "Fusionando cuantización MXFP8 y
     NVFP4": the forward emits its output's amax, the backward the amax of the Hadamard
     rotation of its transposed output).  Nullable device float, 4-byte aligned, raised
     (atomic max) by the call, so the caller sets it to 0 (or a running max) first:
       moe_group_gemm_glu_fwd(_mx): max |y| over the routed rows, bf16 values as written;
       moe_group_gemm_dglu_bwd:     max |R d| over every column d of dgu = [dg | du] (bf16
         values as written) cut into runs of 16 consecutive rows that restart at each group's
         first row, the last run of a group padded with zero rows, and R = H16 S / 4: H16 the
         Sylvester Hadamard matrix of order 16 and S = diag(s_i), s_i = -1 where bit i of
         rht_signs is set (row i of the run), else +1.
     NaN values are skipped.  Other entry points ignore both fields. */
  float* amax_out;
  uint32_t rht_signs;       /* low 16 bits: the row signs of the backward rotation */
  /* Gradients of the epilogue's own parameters, written by moe_group_gemm_dglu_bwd only
     (nullable device fp32 buffers, 4-byte aligned, ADDED to atomically, so the caller zeroes
     them or passes running sums; the summation order is unspecified):
       dbias_out      [E][2I], plain (gate | up) order: per expert, the sum over its rows of
                      dgu (the bf16 values as written) = dL/d(bias) of the FC1 + GLU forward;
       drow_scale_out [M_cap]: for every routed row r, sum over j < I of G[r][j] a(g_c) u_c,
                      G = dY2 W2^T (= dL/dy) and a(g_c) u_c the unscaled GLU output in fp32 =
                      dL/d(row_scale[r]); rows past the routed ones are not touched. */
  float* dbias_out;
  float* drow_scale_out;
} moe_epilogue_t;

/* MXFP8 outputs ([BLOG] "Fusionando cuantización MXFP8 y NVFP4": the
 * quantised activation plus a transposed copy for back prop).  Blocks of 32
 * values share one E8M0 scale X = 2^E, E the smallest integer with
 * amax/X <= 448; elements are e4m3fn(v / X), round-to-nearest-even.
 * For an output of R = M_cap rows and C columns:
 *   row_q [R][C], row_s [R][C/32]          blocks along a row
 *   col_q [C][R], col_s [C][ceil(R/32)+E]  blocks of 32 rows of one column
 *                                          that restart at each group's first
 *                                          row; group e's scales start at column
 *                                          sum_{j<e} ceil(m_j/32)
 * Any pointer may be NULL (that copy is skipped); row_q/row_s and col_q/col_s
 * go in pairs.  No alignment requirement (col_blocked = 1: 16 bytes).
 * e5m2 = 1 selects OCP e5m2 elements instead (the gradient format of an
 * MXFP8 recipe: largest value 57344 = 1.75 * 2^15, the scale rule with 57344
 * in place of 448); 0 = e4m3fn.
 * col_blocked = 1 writes the transposed copy in the K-tiled layout that the
 * MXFP8 weight-gradient GroupGemm (moe_group_gemm_wgrad_mx) reads, the copy
 * the pages keep "for back prop": a row of col_s has S = 4 (ceil(R/128) + E)
 * slots and the matching row of col_q 32 S bytes, slot s holding one 32-row
 * block (its scale byte at col_s[c][s], its 32 codes at col_q[c][32 s ..]);
 * group e's blocks take slots so_e, so_e + 1, ... with so_e = 4 sum_{j<e}
 * ceil(m_j/128), so every group starts on a 128-code boundary, and the slots
 * up to so_e + 4 ceil(m_e/128) that no row reaches (and the codes of a partial
 * block past the group's last row) hold zero codes with scale byte 127.
 * col_blocked = 0 is the dense layout above.  (host struct) */
typedef struct {
  uint8_t* row_q;
  uint8_t* row_s;
  uint8_t* col_q;
  uint8_t* col_s;
  int32_t e5m2;
  int32_t col_blocked;
} moe_mx_out_t;

/* Expert groups.  The counts are the ONLY copy of the group sizes and stay in
 * device memory ([BLOG] "Eliminando la sincronización host-device": tokens
 * per group are tracked in GPU memory, so no host sync is needed and a whole
 * iteration can be captured in a graph).  (host struct) */
typedef struct {
  const int32_t* counts;    /* device [E] */
  int32_t E;                /* 1 <= E <= 1024 */
  int32_t M_cap;            /* static row capacity of every grouped operand */
  int32_t* offsets_out;     /* nullable device [E+1]: exclusive scan of the clamped counts */
  int32_t* status_out;      /* nullable device word, OR-ed: bit0 a count < 0, bit1 sum > M_cap */
} moe_groups_t;

/* Operand descriptor of moe_group_gemm_quant. */
typedef enum {
  MOE_DT_BF16 = 0,
  MOE_DT_MXFP8 = 1,         /* e4m3fn bytes + E8M0 scales, 32-blocks along K */
  MOE_DT_MXFP8_E5M2 = 2,    /* e5m2 bytes + E8M0 scales (a gradient, e.g. dgu for dX); the A operand
                               of moe_group_gemm_quant, either operand of moe_group_gemm_wgrad_mx */
  MOE_DT_MXFP4 = 3,         /* e2m1 codes, two per byte (the lower nibble first), + E8M0 scales,
                               32-blocks along K: see moe_mxfp4_quantize; either operand of
                               moe_group_gemm_quant */
  MOE_DT_FP32 = 4           /* logits of the router; no GEMM operand */
} moe_dtype_t;

typedef enum {
  MOE_B_KN = 0,             /* B_e is [K][N] row-major (N contiguous), e.g. W2 [E][I][H] for FC2 */
  MOE_B_NK = 1,             /* B_e is stored [N][K] (K contiguous), i.e. used transposed:
                               out = A . B_e^T, e.g. W2 [E][I][H] in the dgrad dY2 . W2^T */
  MOE_B_PACKED = 2          /* B_e in the tile-blocked layout of moe_pack_weight (see there) */
} moe_b_layout_t;

typedef struct {
  int32_t dtype;            /* moe_dtype_t */
  int32_t layout;           /* A: ignored (always [M_cap][K] row-major); B: moe_b_layout_t */
  const void* data;         /* bf16 or e4m3 elements */
  const uint8_t* scales;    /* MXFP8 and MXFP4: A [M_cap][K/32] E8M0 (block b of row r covers K
                               values 32b..32b+31); MXFP8 B from moe_pack_weight_mx; MXFP4 B
                               [E][N][K/32] */
} moe_operand_t;

/* Reads the device's compute-unit count once; call before graph capture.
 * Every other call initialises lazily on first use.  The persistent grid of
 * every GroupGemm is sized from that count ([BLOG] "Eliminando la
 * sincronización host-device": a fixed launch whose work split is decided on
 * the device, so the launch itself needs no host-side information that
 * changes between steps). */
moe_status_t moe_init(int device);

const char* moe_status_string(moe_status_t s);

/* Tile-blocked weight layout ("packed"), shared by moe_repack_gate_up and
 * moe_pack_weight.  A weight used as the B operand of out = A . B_e^T is
 * viewed per expert as [N][K] (K contiguous).  It is stored as blocks of 256
 * rows (n) by 64 columns (k) = 32 KiB each; block (nb, kb) starts at element
 * (nb * K/64 + kb) * 16384 of the expert, and experts are ceil(N/256) * 256 * K
 * elements apart.  Inside a block, the 16-byte chunk c (0..7, k = 64 kb + 8c
 * .. +7) of row r (n = 256 nb + r) sits at byte r * 128 + 16 * (c XOR s(r)),
 * s(r) = (r mod 8) XOR (2 ((r / 8) mod 2) + (r / 16) mod 2): the order in
 * which the kernels stage it in LDS, so each block streams from memory
 * contiguously.  Rows n >= N are zero.  Requires K % 64 == 0. */
size_t moe_packed_weight_bytes(int E, int N, int K);

/* Packs per-expert weights into the tile-blocked layout above: the same
 * offline weight preparation as the gate/up repack ([BLOG] "Optimizando GLU
 * vía epílogos GEMM fusionados", Figure 2: the weights are rearranged once, off
 * the training step, into the order the kernel consumes), here without the
 * gate/up interleave, for the other GroupGemm operands.
 * src_layout MOE_B_NK: src is [E][N][K]; MOE_B_KN: src is [E][K][N] (transposed
 * while packing).  Uses: FC2's W2 [E][I][H] as MOE_B_KN with N = H, K = I;
 * dgrad's W2 [E][I][H] as MOE_B_NK with N = I, K = H; dX's plain W1 [E][H][2I]
 * as MOE_B_NK with N = H, K = 2I.  Bit-exact (a permutation plus zero padding). */
moe_status_t moe_pack_weight(const void* src, int E, int N, int K, int src_layout, void* dst,
                             void* stream);

/* MXFP8 weight for the block-scaled GroupGemm ([BLOG] "Fusionando
 * cuantización MXFP8…": MXFP8 blocks of 32 values with one E8M0 scale; here a
 * weight quantised once, offline, along the reduction dimension K).
 * Element bytes: per expert ceil(N/256) * 256 * K (e4m3fn codes), as blocks
 * of 256 rows (n) by 128 K values = 32 KiB; block (nb, kb) starts at byte
 * (nb * K/128 + kb) * 32768 of the expert; the 16-byte chunk c (0..7, k =
 * 128 kb + 16 c .. +15) of row r sits at byte r * 128 + 16 * (c XOR s(r)),
 * s(r) as above.  Scale bytes: per expert ceil(N/256) * 256 * K/32; the
 * dword at byte ((nb * K/128 + kb) * 256 + r) * 4 holds the E8M0 scales of
 * row r's four 32-blocks of block (nb, kb), block b in byte b.  Rows n >= N
 * are zero with scale byte 0.  Requires K % 128 == 0. */
size_t moe_packed_mx_weight_bytes(int E, int N, int K);
size_t moe_packed_mx_scale_bytes(int E, int N, int K);

/* Quantises a bf16 weight to that MXFP8 layout: for each output column n and
 * each run of 32 consecutive k, amax gives the E8M0 exponent X (the smallest
 * power of two with amax / 2^X <= 448; 0xFF if a value is NaN) and every
 * value becomes e4m3fn(v / 2^X), rounded to nearest even.  src_layout as for
 * moe_pack_weight (FC2's W2 [E][I][H]: MOE_B_KN with N = H, K = I).
 * Requires N % 64 == 0, K % 128 == 0; dst_q, dst_s 16-byte aligned. */
moe_status_t moe_pack_weight_mx(const void* src, int E, int N, int K, int src_layout,
                                void* dst_q, void* dst_s, void* stream);

/* The gate/up-repacked W1 as MXFP8 (the FC1 weight of the MXFP8 recipe):
 * W1 [E][H][2I] bf16 (plain: gate | up) quantised along H (the reduction
 * dimension) and stored in the MXFP8 layout above with N = 2I in the packed
 * gate/up order of moe_repack_gate_up and K = H.  Sizes:
 * moe_packed_mx_weight_bytes(E, 2I, H), moe_packed_mx_scale_bytes(E, 2I, H).
 * Requires H % 128 == 0, I % 64 == 0. */
moe_status_t moe_repack_gate_up_mx(const void* w1, int E, int H, int I, void* dst_q, void* dst_s,
                                   void* stream);

/* Bytes of the packed W1 for E experts, hidden H, intermediate I:
 * moe_packed_weight_bytes(E, 2I, H). */
size_t moe_packed_w1_bytes(int E, int H, int I);

/* Offline gate/up repack ([BLOG] "Optimizando GLU…" and its Figure 2: W1's
 * columns are repacked into interleaved gate and input (up) blocks so that one
 * GEMM tile holds half a tile width of each; done once at checkpoint load).
 * w1:        bf16 [E][H][2I], plain: columns [0,I) gate, [I,2I) up.
 * w1_packed: the tile-blocked layout above with N = 2I (packed order), K = H,
 *            where packed row 128p + s is gate column 64p + s for s < 64 and up
 *            column I + 64p + (s-64) for s >= 64.  Each 256-row block therefore
 *            holds two (64 gate | 64 up) pairs.  Requires I % 64 == 0,
 *            H % 64 == 0.  Bit-exact. */
moe_status_t moe_repack_gate_up(const void* w1, int E, int H, int I, void* w1_packed,
                                void* stream);

/* Inverse of moe_repack_gate_up (checkpoint save, tests).  Bit-exact. */
moe_status_t moe_unpack_gate_up(const void* w1_packed, int E, int H, int I, void* w1,
                                void* stream);

/* Device routing and grouping ([MEGA] §2.1: each token's k experts are the
 * k largest router logits; §4.3: rows of one expert laid out contiguously).
 * Exactly one of logits (fp32 [T][E]) / topk_ids (int32 [T][k]) is non-NULL.
 * Ties go to the lower expert id.  Outputs (all device, all required except
 * xg): topk_ids_out [T][k]; counts [E]; offsets [E+1]; dst [T][k], the grouped
 * row of pair (t, j); src [T*k], the token of each grouped row.  Within an
 * expert the pairs keep ascending (t, j) order, so the result is unique and
 * deterministic.  If x (bf16 [T][H]) and xg (bf16 [T*k][H]) are given, xg
 * receives the gathered rows xg[r] = x[src[r]].  Given topk_ids outside
 * [0, E) are not grouped: their dst entries and the rows of xg from
 * offsets[E] on are left as they were, and src entries from offsets[E] on are
 * set to -1.  Requires k <= E <= 1024, k <= 16,
 * T*k < 2^31, H % 8 == 0. */
moe_status_t moe_route_group(const float* logits, const int32_t* topk_ids, int T, int E, int k,
                             int32_t* topk_ids_out, int32_t* counts, int32_t* offsets,
                             int32_t* dst, int32_t* src, const void* x, int H, void* xg,
                             void* stream);

/* GroupGemm + Activation (+ Quantize/Transpose), the fused FC1 ([BLOG] kernel
 * family, second kernel).  For each expert e, with A_e = xg rows of group e:
 *     z = A_e . W1_e (+ bias_e)          fp32 accumulate, W1 from moe_repack_gate_up
 *     preact = bf16(z)                   optional, [M_cap][2I] in PLAIN order
 *     y = bf16(GLU epilogue of z)        optional, [M_cap][I]
 *     mx = MXFP8 copies of y             optional (row-wise and/or transposed)
 * xg: bf16 [M_cap][H]; w1_packed from moe_repack_gate_up.
 * Non-gated form (ep->gated == 0): W1 [E][H][I] packed by moe_pack_weight
 * (MOE_B_KN source, N = I, K = H), z and preact are [M_cap][I], y = bf16(a(z)
 * * row_scale); bias [E][I].
 * Requires H % 64 == 0, I % 64 == 0.
 * One persistent launch; tiles are scheduled from the device counts.
 * cu_margin: compute units left free for concurrent kernels (0 = use all). */
moe_status_t moe_group_gemm_glu_fwd(const void* xg, const moe_groups_t* groups,
                                    const void* w1_packed, int H, int I,
                                    const moe_epilogue_t* ep, void* y, void* preact,
                                    const moe_mx_out_t* mx, int cu_margin, void* stream);

/* moe_group_gemm_glu_fwd with MXFP8 inputs ([BLOG] "Fusionando cuantización
 * MXFP8…": the MXFP8 training recipe's FC1): xg = e4m3 [M_cap][H] with E8M0
 * row-block scales [M_cap][H/32] (e.g. moe_mxfp8_quantize of the bf16 rows),
 * w1 = MOE_B_PACKED from moe_repack_gate_up_mx.  z is accumulated in fp32 by
 * the block-scaled MFMA from the dequantised operands; the epilogue and the
 * outputs are those of moe_group_gemm_glu_fwd.  Requires H % 128 == 0,
 * I % 64 == 0. */
moe_status_t moe_group_gemm_glu_fwd_mx(const moe_operand_t* xg, const moe_groups_t* groups,
                                       const moe_operand_t* w1, int H, int I,
                                       const moe_epilogue_t* ep, void* y, void* preact,
                                       const moe_mx_out_t* mx, int cu_margin, void* stream);

/* GroupGemm + dActivation (+ Quantize/Transpose), the fused backward of FC1's
 * activation ([BLOG] "Optimizando GLU…": in back prop the epilogue reads the
 * GEMM output, computes the dGLU and writes it out).  Per expert:
 *     G = dy2_e . W2_e^T                 fp32 accumulate; dy2 bf16 [M_cap][H];
 *                                        w2: FC2's weight [E][I][H] bf16 as
 *                                        MOE_B_NK, or moe_pack_weight of it
 *                                        (MOE_B_NK source, N = I, K = H) as
 *                                        MOE_B_PACKED
 *     with g, u from preact (bf16 [M_cap][2I] plain, post-bias, pre-clamp),
 *     gc = clamp(g), uc = clamp(u) + up_offset, rs = row_scale or 1:
 *     du = G * a(gc) * rs * [up_lo <= u <= up_hi]
 *     dg = G * uc * rs * a'(gc) * [gate_lo <= g <= gate_hi]
 *     dgu = bf16([dg | du])              [M_cap][2I] plain order
 *     mx = MXFP8 copies of dgu           optional
 * Non-gated form (ep->gated == 0): preact and dgu are [M_cap][I] and
 * dgu = bf16(G * rs * a'(z)); the parameter gradients are not available
 * (MOE_ERR_UNSUPPORTED), the rotated amax is.
 * ep->bias is ignored (already inside preact).  Requires H % 64 == 0,
 * I % 64 == 0. */
moe_status_t moe_group_gemm_dglu_bwd(const void* dy2, const moe_operand_t* w2, int H, int I,
                                     const moe_groups_t* groups, const void* preact,
                                     const moe_epilogue_t* ep, void* dgu,
                                     const moe_mx_out_t* mx, int cu_margin, void* stream);

/* GroupGemm + Quantize ([BLOG] kernel family, first kernel): out_e = A_e . B_e
 * with bf16 and/or MXFP8 output.  A: [M_cap][K] grouped rows; B per the
 * layout in b->layout (MOE_B_PACKED is the fast path).  c_bf16: nullable bf16
 * [M_cap][N].  bf16 x bf16 on every B layout, or MXFP8 x MXFP8 ([BLOG]
 * "GroupGemm + Quantize" with MXFP8 inputs): A = e4m3fn [M_cap][K] with E8M0
 * row-block scales [M_cap][K/32] (e.g. the row-wise MX output of
 * moe_group_gemm_glu_fwd), B = MOE_B_PACKED from moe_pack_weight_mx, and
 *     out_e = sum_k (q_a * 2^(s_a - 127)) (q_b * 2^(s_b - 127))
 * accumulated in fp32 by the block-scaled MFMA.  Mixed bf16 / MXFP8 inputs
 * are MOE_ERR_UNSUPPORTED.  Requires K % 64 == 0 (K % 128 == 0 for MXFP8),
 * N % 64 == 0.
 * MXFP4 weights (4-bit floating point, the weight format of GPT-OSS-like
 * models): B = e2m1 codes [E][N][K/2] in the plain MOE_B_NK layout (K
 * contiguous, the layout such checkpoints hold) with E8M0 scales [E][N][K/32],
 * e.g. from moe_pack_weight_mxfp4; A = e2m1 codes [M_cap][K/2] (MOE_DT_MXFP4,
 * moe_mxfp4_quantize) or e4m3fn codes [M_cap][K] (MOE_DT_MXFP8), with scales
 * [M_cap][K/32]: the same sum over the codes' values.  4-bit rows are summed to
 * fp32's rounding; with 8-bit rows, as in the MXFP8 products, the MFMA cuts
 * products off below the largest of the 64 that it adds (within 2^-11.8 of it),
 * so that a few outputs in a thousand are a bf16 step off.  A scale byte 0xFF (NaN)
 * makes every product with its block NaN.  c_bf16 is required, MXFP8 outputs
 * are MOE_ERR_UNSUPPORTED.  Requires K % 32 == 0, K < 2^24, N % 64 == 0, N <
 * 2^23; codes and c 16-byte aligned, scales any.  The call takes any group
 * sizes, from one row per expert (decoding, where it streams the active
 * experts' weights once) up; which of its kernels runs goes by M_cap, since
 * the host does not know the counts, so a decoding batch is best given the
 * capacity that it can fill. */
moe_status_t moe_group_gemm_quant(const moe_operand_t* a, const moe_operand_t* b, int N, int K,
                                  const moe_groups_t* groups, void* c_bf16,
                                  const moe_mx_out_t* mx, int cu_margin, void* stream);

/* Weight gradients as K-grouped GroupGemms ([BLOG] "Fusionando cuantización
 * MXFP8…": the transposed copies exist for back prop, i.e. for these
 * products).  For each expert e with rows [o_e, o_e + m_e):
 *     c_e = a_e^T . b_e          fp32 accumulate, fp32 output [E][P][Q]
 * a: bf16 [M_cap][P] grouped rows, b: bf16 [M_cap][Q] grouped rows; the
 * reduction runs over the group's rows (counts in device memory only).
 * dW1 = wgrad(xg [M_cap][H], dgu [M_cap][2I]) -> [E][H][2I] (plain W1 order);
 * dW2 = wgrad(y [M_cap][I], dy2 [M_cap][H]) -> [E][I][H].
 * accumulate = 0 overwrites c (an empty group writes zeros); 1 adds to it.
 * Requires P % 64 == 0, Q % 64 == 0; a, b, c 16-byte aligned. */
moe_status_t moe_group_gemm_wgrad(const void* a, const void* b, int P, int Q,
                                  const moe_groups_t* groups, float* c, int accumulate,
                                  int cu_margin, void* stream);

/* MXFP8 weight gradients ([BLOG] "Fusionando cuantización MXFP8 y NVFP4": the
 * epilogues also write a transposed MXFP8 copy "for back prop"; these are
 * the products that read it): the same K-grouped GroupGemm as
 * moe_group_gemm_wgrad, C_e = A_e^T B_e in fp32 [E][P][Q], on the
 * block-scaled MFMA, each operand a transposed MXFP8 copy in the K-tiled
 * layout of moe_mx_out_t (col_blocked = 1) over the same groups:
 *   a->data  [P][32 S] codes, a->scales [P][S] E8M0 (the col_q/col_s of an
 *            [M_cap][P] tensor), S = 4 (ceil(M_cap/128) + E);
 *   b->data  [Q][32 S], b->scales [Q][S] likewise;
 *   dtype    MOE_DT_MXFP8 (e4m3 codes) or MOE_DT_MXFP8_E5M2, per operand;
 *            layout ignored.
 * The result is the exact product of the dequantised copies up to fp32
 * accumulation: dW1 from the copies of xg and dgu, dW2 from those of y and
 * dy2.  accumulate = 0 overwrites c (an empty group writes zeros); 1 adds.
 * Requires P % 64 == 0, Q % 64 == 0; codes and c 16-byte aligned, scales
 * 4-byte aligned. */
moe_status_t moe_group_gemm_wgrad_mx(const moe_operand_t* a, const moe_operand_t* b, int P, int Q,
                                     const moe_groups_t* groups, float* c, int accumulate,
                                     int cu_margin, void* stream);

/* Unfused GLU pass ([BLOG] "¿Dónde se va el cómputo en un bloque MoE?": the
 * activation as its own memory-bound pass between the GEMMs, the baseline the
 * fused epilogue replaces): y = GLU epilogue of z, where z is
 * the plain-order bf16 [M_cap][2I] FC1 output WITHOUT bias (bias, if any, is
 * added here).  Same arithmetic as the fused epilogue, as its own kernel. */
moe_status_t moe_glu_unfused(const void* z, const moe_groups_t* groups, int I,
                             const moe_epilogue_t* ep, void* y, void* stream);

/* Unfused dGLU pass (the baseline of the fused backward epilogue, [BLOG]
 * "Optimizando GLU vía epílogos GEMM fusionados": the activation gradient as a
 * memory-bound pass after the GEMM).  g: dL/dy bf16 [M_cap][I] as the plain
 * dgrad GroupGemm wrote it (moe_group_gemm_quant of dY2 with W2); z: the saved
 * pre-activation bf16 [M_cap][2I] (plain order, post-bias); dgu: bf16
 * [M_cap][2I] output, d(gate) in columns [0, I), d(up) in [I, 2I).  Same
 * arithmetic as moe_group_gemm_dglu_bwd's epilogue (row scale, clamp
 * gradients, activation derivative) on the bf16-rounded g.  Routed rows only
 * (offsets from the device counts); gated forms only (ep->gated = 1, else
 * MOE_ERR_UNSUPPORTED).  Requires I % 64 == 0; g, z, dgu 16-byte aligned. */
moe_status_t moe_dglu_unfused(const void* g, const void* z, const moe_groups_t* groups, int I,
                              const moe_epilogue_t* ep, void* dgu, void* stream);

/* Standalone MXFP8 quantize/transpose ([BLOG] "Fusionando cuantización MXFP8 y
 * NVFP4": the separate pass that reads the bf16 activation output and writes
 * the MXFP8 copy and its transposed version, which the fused epilogues
 * replace; also the offline weight prep) of
 * a bf16 [R][C] matrix.  Row-wise blocks run along C.  Column-wise blocks run
 * down 32 rows; with groups (counts over the first rows, M_cap = R) they
 * restart at each group's first row exactly as in the fused epilogues and
 * col_s is [C][ceil(R/32)+E]; without groups the whole matrix is one group
 * and col_s is [C][ceil(R/32)].  So quantising one expert's W2_e [I][H]
 * column-wise yields exactly the [H][I] e4m3 + [H][I/32] scale operand that
 * MOE_B_NK expects.  Requires C % 32 == 0. */
moe_status_t moe_mxfp8_quantize(const void* v, int R, int C, const moe_groups_t* groups,
                                const moe_mx_out_t* mx, void* stream);

/* The operators around the GEMMs: the calls below and moe_group_gemm_quant with
 * MXFP4 weights.  An output may not share bytes with an input or with another
 * output, but where a call says that it may be the same buffer
 * (MOE_ERR_UNSUPPORTED otherwise).  An array without rows (of T = 0 tokens, of
 * M_cap or R = 0 rows) may be NULL, as an empty tensor's address is. */

/* Router ([MEGA] §2.1: scores p = Softmax(W_r x), the k best experts of each
 * token, and their scores as the weights of the expert outputs).  From a
 * token's logits x [E]:
 *   s_e = softmax(x)_e or sigmoid(x_e)                       the scores
 *   c_e = s_e + bias_e                                       the choice values
 * bias is a balance term for the choice alone (an offset that training moves
 * up for underused experts): the weights are the scores without it.  Without a
 * bias the experts are ordered by their logits, which is the same order.
 * n_groups > 1: the experts form n_groups groups of E / n_groups consecutive
 * ids; a group's value is its best choice value (MOE_GROUP_MAX) or the sum of
 * its two best (MOE_GROUP_TOP2; without a bias of its two best scores), and
 * only the topk_groups best groups take part.  The k largest choice values
 * are taken, in that order; ties go to the lower id, of groups too, and the
 * choice is made in 64 bits.  With S = the sum of the chosen scores (renorm =
 * 1) or 1 (renorm = 0):
 *   w_j = scale * s_j / S
 * NaN logits (and choice values) rank below every number; a NaN logit makes
 * the softmax of its row NaN.  Where S is 0 (the scores taken in 64 bits: a
 * softmax's below about e^-745 of the row's best, a sigmoid's of logits below
 * -709), or every logit of a softmax row is -inf, the weights are 0.  (host
 * struct) */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_t;
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 } moe_group_score_t;
typedef struct {
  int32_t score;            /* moe_score_t */
  int32_t n_groups;         /* 1 .. 64, divides E; 1 = no groups */
  int32_t topk_groups;      /* 1 .. n_groups */
  int32_t group_score;      /* moe_group_score_t */
  int32_t renorm;           /* 1: weights divided by their sum */
  float scale;              /* finite; multiplies the weights */
  const float* bias;        /* nullable device fp32 [E] */
} moe_router_t;

/* ids [T][k] int32 and weights [T][k] fp32 from logits [T][E] (fp32:
 * MOE_DT_FP32, or MOE_DT_BF16).  The ids feed moe_route_group (as topk_ids),
 * the weights moe_combine (or, grouped, the epilogue's row_scale).  Requires
 * 1 <= k <= 16, k <= E <= 1024, k <= topk_groups * E / n_groups (groups of at
 * least 2 experts for MOE_GROUP_TOP2), T <= 2^25; logits 16-byte, ids, weights
 * and bias 4-byte aligned.  T = 0 does nothing, here and below. */
moe_status_t moe_router_topk(const void* logits, int logits_dtype, int T, int E, int k,
                             const moe_router_t* router, int32_t* ids, float* weights, void* stream);

/* Gradient of the router's weights: dlogits [T][E] (the logits' type) from
 * dweights [T][k] fp32, for the ids that moe_router_topk chose from the same
 * logits (the choice itself and the bias have no gradient).  Every entry of
 * dlogits is written.  Ids outside [0, E) take no part; an id that stands
 * twice in a token counts twice.  Where the weights are 0 by the rule above,
 * so is the gradient.  A renormalised softmax is the softmax over the chosen
 * logits and has no gradient at others (which are read only with a bias or
 * MOE_GROUP_TOP2, to see whether S is 0).  dlogits 16-byte aligned, else as above. */
moe_status_t moe_router_topk_bwd(const void* logits, int logits_dtype, int T, int E, int k,
                                 const moe_router_t* router, const int32_t* ids, const float* dweights,
                                 void* dlogits, void* stream);

/* Combine ([MEGA] §2.1: y = E_shared(x) + sum_j p_j E_j(x)): a token's expert
 * rows back to the token,
 *   out[t] = residual[t] + sum_{j < k} weights[t][j] y[dst[t][j]]
 * added in slot order in fp32 and rounded once to bf16.  y: bf16 [M_cap][H]
 * grouped rows (FC2's output), dst [T][k] from moe_route_group (a pair whose
 * dst lies outside [0, M_cap) adds nothing: preset dst to -1 if ids may be
 * dropped), weights fp32 [T][k] (NULL: all 1, which makes this call the
 * gradient of the row gather), residual bf16 [T][H] (NULL: none; the shared
 * expert's output or the residual stream), out bf16 [T][H], which may be the
 * residual itself.  Requires H % 8 == 0, H <= 2^26, 1 <= k <= 16; y, residual
 * and out 16-byte, dst and weights 4-byte aligned. */
moe_status_t moe_combine(const void* y, int M_cap, int H, const int32_t* dst, const float* weights, int T,
                         int k, const void* residual, void* out, void* stream);

/* Gradients of moe_combine (the residual's is dout itself):
 *   dy[dst[t][j]] = bf16(weights[t][j] dout[t])      bf16 [M_cap][H], nullable
 *   dweights[t][j] = sum_h dout[t][h] y[dst[t][j]][h]  fp32 [T][k], nullable
 * with 0 in dweights for a pair without a row.  Rows of dy that no pair names
 * are not written.  A row belongs to one token (as moe_route_group's do); if
 * two slots of a token name it, it gets the sum of their gradients.  y is
 * needed for dweights only. */
moe_status_t moe_combine_bwd(const void* dout, const void* y, int M_cap, int H, const int32_t* dst,
                             const float* weights, int T, int k, void* dy, float* dweights, void* stream);

/* Residual addition + root-mean-square norm, the pass in front of the expert
 * MLP, with the MXFP8 rows that its GEMMs read:
 *   h = bf16(x + residual)                 residual NULL: h = x
 *   rstd = 1 / sqrt(mean(h^2) + eps)       per row, fp32
 *   y = bf16(h * rstd * weight)
 *   mx: row-wise MXFP8 copy of y (mx->row_q, row_s; byte-identical to
 *       moe_mxfp8_quantize of y; the transposed copy is MOE_ERR_UNSUPPORTED)
 * x, residual, h, y: bf16 [T][H]; weight bf16 [H]; rstd fp32 [T].  Each output
 * may be NULL, one is required.  h may be x or residual itself.  Requires H %
 * 8 == 0, 8 <= H <= 16384 (H % 32 == 0 with mx), eps >= 0; x, residual, weight,
 * h and y 16-byte, rstd 4-byte aligned. */
moe_status_t moe_add_rmsnorm(const void* x, const void* residual, const void* weight, int T, int H,
                             float eps, void* h, void* y, float* rstd, const moe_mx_out_t* mx, void* stream);

/* Its gradients from dy (bf16 [T][H]), the saved h and rstd, and dh (bf16
 * [T][H], nullable: the gradient that reaches h past the norm).  With n = h
 * rstd and g = dy weight:
 *   dx = bf16(rstd (g - n mean(g n)) + dh)   bf16 [T][H], nullable: the
 *                                            gradient of x and of residual
 *   dweight = sum_t dy n                     fp32 [H], nullable; accumulate = 1
 *                                            adds to it (T = 0: sets it to 0,
 *                                            or adds nothing)
 * dweight needs the workspace (moe_add_rmsnorm_bwd_workspace_bytes(T, H)
 * bytes, 16-byte aligned, contents of no meaning before or after; calls that
 * may run at the same time, replays of captured ones too, need one each); its
 * sums are added in a fixed order.  dx may be dh itself. */
size_t moe_add_rmsnorm_bwd_workspace_bytes(int T, int H);
moe_status_t moe_add_rmsnorm_bwd(const void* dy, const void* h, const void* weight, const float* rstd,
                                 const void* dh, int T, int H, void* dx, float* dweight, int accumulate,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* MXFP4 quantisation of a bf16 [R][C] matrix along its rows (OCP MX: blocks
 * of 32 values, one E8M0 scale X = 2^E, E the smallest integer with amax/X <=
 * 6, the largest e2m1 value, as moe_mx_out_t's rule has it for 448; elements
 * e2m1(v / X), round-to-nearest-even):
 *   q [R][C/2]: value c of a row in byte c / 2, the lower nibble for even c
 *   s [R][C/32] E8M0
 * A block holding a NaN or an infinity gets scale 0xFF (NaN) and zero codes.
 * With groups (M_cap = R) only the routed rows are read and written.  Requires
 * C % 32 == 0; v and q 16-byte aligned. */
moe_status_t moe_mxfp4_quantize(const void* v, int R, int C, const moe_groups_t* groups, uint8_t* q,
                                uint8_t* s, void* stream);

/* Offline MXFP4 quantisation of a bf16 weight along its reduction dimension
 * K, into the plain MOE_B_NK layout that moe_group_gemm_quant reads: dst_q
 * [E][N][K/2], dst_s [E][N][K/32].  src_layout MOE_B_NK: src is [E][N][K];
 * MOE_B_KN: src is [E][K][N] (FC1's plain W1 [E][H][2I]: N = 2I, K = H; FC2's
 * W2 [E][I][H]: N = H, K = I).  Requires N % 64 == 0, K % 32 == 0, E <= 65535,
 * E * N < 2^31. */
moe_status_t moe_pack_weight_mxfp4(const void* src, int E, int N, int K, int src_layout, void* dst_q,
                                   void* dst_s, void* stream);

/* Low-rank adapters of many requests beside a shared projection: for the rows
 * of group e (moe_groups_t: counts [E], one group per adapter, or per expert)
 *   u_i = A_e x_i                         fp32, the narrow product
 *   y_i = bf16(base_i + scale_e B_e u_i)
 * A bf16 [E][r][K] and B bf16 [E][N][r] as such adapters are stored, scale fp32
 * [E] (alpha / r; NULL: 1).  Adapters of a smaller rank are padded with zeros.
 * x_ld, y_ld: elements from one row of x (and dx) and of y (base, dy) to the
 * next, 0 = K and N; more than that for columns of a wider matrix.  Requires r
 * % 8 == 0, 8 <= r <= 128, K and N % 8 == 0, 8 <= K, N <= 2^17, x_ld >= K and
 * y_ld >= N multiples of 8, x_ld and y_ld <= 2^32 and T rows of them within
 * 2^48 elements.  (host struct) */
typedef struct {
  const void* A;
  const void* B;
  const float* scale;       /* nullable */
  int32_t r, K, N;
  int64_t x_ld, y_ld;
} moe_lora_t;

/* The adapters' products onto the shared projection's output.  x: bf16 [T][K],
 * base, y: bf16 [T][N] (base NULL: 0; y may be base itself).  src int32 [M_cap]
 * names the row of x and y that a grouped row is, as moe_route_group's src does
 * (adapter ids as topk_ids, k = 1; one grouping serves every projection of a
 * step), NULL: the grouped row itself; no row stands in it twice.  Rows that no
 * group holds, and grouped rows whose src lies outside [0, T), are left as they
 * were.  u: fp32 [M_cap][r] or NULL, kept for the backward pass (0 in rows whose
 * src lies outside).  All sums are fp32; the product with B takes u to 2^-17 of
 * its value, in two parts, so that an infinity of B may give NaN.  workspace:
 * moe_lora_fwd_workspace_bytes(M_cap, E, r, K, N) bytes (0 where one launch does
 * it: few rows of a small adapter; then NULL will do), 16-byte aligned, contents
 * of no meaning before or after; calls that may run at the same time, replays of
 * captured ones too, need one each.  Requires M_cap <=
 * 2^25; x, A, B, base, y, u 16-byte, src and scale 4-byte aligned.  T = 0 does
 * nothing but report the groups. */
size_t moe_lora_fwd_workspace_bytes(int M_cap, int E, int r, int K, int N);
moe_status_t moe_lora_fwd(const void* x, int T, const int32_t* src, const moe_groups_t* groups,
                          const moe_lora_t* lora, const void* base, void* y, float* u, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Its gradients from dy (bf16 [T][N]) and the saved u, with w_i = B_e^T dy_i:
 *   dx_i = bf16(dx_base_i + scale_e A_e^T w_i)      bf16 [T][K], nullable; dx may
 *                                                   be dx_base itself (NULL: 0)
 *   dA_e = scale_e sum_i w_i x_i^T                  fp32 [E][r][K], nullable
 *   dB_e = scale_e sum_i dy_i u_i^T                 fp32 [E][N][r], nullable
 * dy has y's row distance, dx and dx_base x's.  accumulate = 1 adds to dA and
 * dB; 0 writes them (0 for a group without rows; T = 0 too).  x is needed for dA
 * only, u for dB only.  Sums are fp32, in a fixed order; an infinity of A (for
 * dx), of x (for dA) or of dy (for dB) may give NaN.  The workspace (of
 * moe_lora_bwd_workspace_bytes) and the rest as above; rows of dx that no group
 * holds are left as they were. */
size_t moe_lora_bwd_workspace_bytes(int M_cap, int E, int r, int K, int N);
moe_status_t moe_lora_bwd(const void* dy, const void* x, int T, const int32_t* src, const moe_groups_t* groups,
                          const moe_lora_t* lora, const float* u, const void* dx_base, void* dx, float* dA,
                          float* dB, int accumulate, void* workspace, size_t workspace_bytes, void* stream);

/* A tensor of an AdamW step: n elements of a parameter, its gradient (e.g. the
 * fp32 dW of moe_group_gemm_wgrad) and its states.
 *   param   fp32 or bf16 (param_dtype MOE_DT_FP32 or MOE_DT_BF16); NULL: the
 *           tensor takes part in moe_grad_norm alone
 *   grad    fp32 or bf16 (grad_dtype)
 *   master  fp32 [n], the value that a bf16 parameter is the rounding of; NULL:
 *           the parameter's own value is updated and rounded (to nearest even,
 *           so that updates below half its step are lost)
 *   m, v    state_bits 32: fp32 [n].  state_bits 8: m int8 [n], v uint8 [n] and
 *           per 128 elements m_scale and v_scale fp32 [ceil(n/128)]:
 *             m = sign(c) (c / 127)^2 m_scale,  sqrt(v) = (c / 255)^2 v_scale
 *           m_scale the block's largest |m|, v_scale its largest sqrt(v).  All
 *           zeros is the state before the first step.
 * param, grad, master, m and v 16-byte, the scales 4-byte aligned.  (host
 * struct) */
typedef struct {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;                /* 0 <= n <= 2^42 */
  float lr_scale;           /* multiplies the step's learning rate */
  float weight_decay;
  int32_t param_dtype;
  int32_t grad_dtype;
  int32_t state_bits;
} moe_adamw_tensor_t;

/* The tensors of a step, laid out once: moe_adamw_plan fills `table` (host
 * memory of moe_adamw_plan_bytes(tensors, n_tensors) bytes, 8-byte aligned) and
 * plan's sizes; the caller copies the table to device memory (16-byte aligned)
 * and sets plan->table.  The plan holds as long as the tensors' addresses do;
 * their contents may change.  (A plan of 300 tensors takes 0.1 ms here, copy
 * apart, and 4 ms from Python, where each tensor's struct is made and checked:
 * gradients that get new memory every step cost a new plan every step, so keep
 * their buffers.)  An output of a tensor (param, master, m, v,
 * scales) that shares bytes with any other buffer of the plan is
 * MOE_ERR_UNSUPPORTED.  Where the call fails the table's contents mean nothing.
 * (host struct) */
typedef struct {
  const void* table;        /* device */
  int64_t n_chunks;         /* pieces of the tensors, as the table lists them */
  int64_t n_chunks8;        /* of them, the last ones: those of tensors with 8-bit states */
} moe_adamw_plan_t;
size_t moe_adamw_plan_bytes(const moe_adamw_tensor_t* tensors, int n_tensors);
moe_status_t moe_adamw_plan(const moe_adamw_tensor_t* tensors, int n_tensors, void* table, size_t table_bytes,
                            moe_adamw_plan_t* plan);

/* The step's numbers.  (host struct) */
typedef struct {
  double lr, beta1, beta2, eps;
  int64_t step;             /* number of this step, from 1; ignored with step_dev */
  const int32_t* step_dev;  /* nullable device int32 (below 1 counts as 1): for captured steps */
  const float* lr_dev;      /* nullable device fp32, in the place of lr */
  const float* grad_scale;  /* nullable device fp32 that multiplies every gradient (moe_grad_norm's
                               factor); where it is NaN the call changes nothing */
} moe_adamw_t;

/* One AdamW step over every tensor of the plan, in one launch for each width of
 * state among them.  With g = grad * grad_scale, a = lr * lr_scale and t the
 * step:
 *   m' = beta1 m + (1 - beta1) g,   v' = beta2 v + (1 - beta2) g^2
 *   p' = p (1 - a weight_decay) - a (m' / (1 - beta1^t)) / (sqrt(v' / (1 - beta2^t)) + eps)
 * in fp32.  8-bit states: m' and v' are formed in 64 bits, p' takes them before
 * they are rounded to codes, and the code is the nearest under the square root
 * (the lower of two as near; at least 1 for v' > 0), scales rounded to fp32.  A
 * block in which m' or v' is not finite gets scales NaN and codes 0.  Requires
 * 0 <= beta < 1, eps >= 0, all finite.
 *
 * What 8-bit states are worth: codes move by whole codes, a v's falls in a step
 * without a gradient only where code (1 - beta2^(1/4)) >= 1/2 (beta2 = 0.99: from
 * 200 on; above (1 - 1/510)^4 = 0.9922 never), else with its block's scale alone,
 * which follows the block's largest v; an m's where code (1 - beta1^(1/2)) >= 1/2
 * (beta1 = 0.9: from 10 on).  sqrt(v) over the true one, fifth to 95th percentile
 * of normally distributed gradients: 0.98 to 1.03 at beta2 = 0.99; at 0.999 0.88
 * to 1.16 where a block's gradients are of uneven size, 0.98 to 1.42 after 4000
 * steps and 1.1 to 1.7 in the end where they are of one size; 2.4 to 3.6 and 7.9
 * to 13.2, 2000 and 6000 steps after its gradients fell tenfold, for an element
 * beside others whose did not.  Its steps are that much too small.  32 bits for
 * tensors whose elements' gradients come and go one by one; a beta2 of 0.99 or
 * less has little of this where gradients are not 0. */
moe_status_t moe_adamw_step(const moe_adamw_plan_t* plan, const moe_adamw_t* hyper, void* stream);

/* 8-bit states read out as fp32 (to save, inspect or widen them): m_out, v_out
 * [n], each nullable with its codes; 16-byte aligned codes and outputs. */
moe_status_t moe_adamw_unpack(const int8_t* m, const float* m_scale, const uint8_t* v, const float* v_scale,
                              int64_t n, float* m_out, float* v_out, void* stream);

/* The norm of all gradients of a plan, and the factor that clips them:
 *   out[0] = sqrt(sum of squares),  out[1] = min(1, max_norm / (out[0] + 1e-6))
 * fp32, from sums in 64 bits in a fixed order; out[1] is NaN where out[0] is not
 * finite, so that a step given it as grad_scale is left out.  max_norm > 0 (inf:
 * no clipping).  workspace: moe_grad_norm_workspace_bytes() bytes, 16-byte
 * aligned, one per call that may run at the same time; out 4-byte aligned. */
size_t moe_grad_norm_workspace_bytes(void);
moe_status_t moe_grad_norm(const moe_adamw_plan_t* plan, float max_norm, float* out, void* workspace,
                           size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GLU_H */
