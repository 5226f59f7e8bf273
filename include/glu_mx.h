/*
 * glu_mx.h - C ABI of the MI355X (gfx950) fused gated-linear-unit library.
 *
 * The library computes a gated linear unit h = act(gate) * up, forward and backward, in
 * FP32 with one BF16 rounding at the store, and can emit the result directly as
 * block-scaled ("microscaling") data in one pass over the inputs:
 *   - MXFP8: E4M3 codes with one E8M0 scale per 32 elements, the scale rounded up
 *     (RCEIL) from the block maximum; rowwise 1x32 blocks, colwise 32x1 blocks, or both.
 *   - NVFP4: E2M1 codes packed two per byte with one E4M3 scale per 16 elements and a
 *     global scale of 1.
 * Activations: SwiGLU, act = silu(x) = x * sigmoid(x); GeGLU, act = gelu_tanh(x) =
 * x/2 * (1 + tanh(sqrt(2/pi) * (x + 0.044715 x^3))); GeGLU with the exact GELU,
 * act = x * Phi(x) (Phi the standard normal CDF); ReLU^2, act = max(x, 0)^2.  The last two
 * go beyond the pages, which plan more activations than SiLU ([MX] Follow-ups)
 * without naming them.
 *
 * Sources, cited by page title and section:
 *   [MX] "Add swiglu + MXFP8 fused CuTe DSL kernel": Summary (swiglu fused with the
 *        RCEIL MXFP8 cast, gate/up read once, rowwise/colwise/both from one pass), API
 *        (gated_input packs [gate | up]; backward returns [dGate | dUp]; a disabled
 *        direction comes back zero-sized), Numerics and tests (the fused result equals
 *        the activation followed by the standalone quantizers; launcher guards for the
 *        32-bit bound, pointer alignment and geometry).
 *   [NV] "feat(phyai-kernel): add Thor NVFP4 GeGLU kernel for pi0.5": Summary (GeGLU fold
 *        and compact NVFP4 store), Supported contract (E2M1 values, E4M3 scales in the
 *        CUTLASS/FlashInfer 128x4 layout, global scale 1, pairwise-interleaved gate/up,
 *        caller-supplied output buffers, unsupported inputs fail before launch).
 *   [GE] "perf: tile wide GeGLU rows on SM103": Summary and Testing Done (GeGLU forward,
 *        da and db; ragged widths such as 8193 columns).
 *   [H]  "[WS1] Add batch-invariant h_aggregate kernel": Fixed numerical paths (one
 *        FP32-to-BF16 conversion at the final store) and Supported profile and
 *        fail-closed behavior (no silent copies, unsupported layouts raise).
 *
 * Conventions shared by every entry point:
 *   - BF16 values are passed as uint16_t bit patterns.  Every data pointer is a device
 *     pointer; the library never dereferences one on the host.
 *   - Extents and row strides ("ld", in elements) are int64_t.  Matrices are row-major.
 *   - Caller-owned buffers: the library never allocates, frees or synchronizes, and keeps
 *     no mutable global state, so calls are thread-safe and can be captured in a HIP
 *     graph.  `stream` is a hipStream_t passed as void*; NULL means the null stream.
 *   - Fail closed: every argument is validated on the host before any HIP call.  On any
 *     status other than GLU_OK nothing was launched and nothing was written.  A kernel
 *     fault surfaces at the caller's next synchronization, not here.
 *   - M == 0 or N == 0 is a valid no-op (pointers are then not inspected).
 *   - Every base pointer must be 16-byte aligned (GLU_ERR_ALIGN).
 *   - Outputs may not overlap inputs or each other (GLU_ERR_OVERLAP), judged on the byte
 *     range each operand spans; the one exception is the in-place backward of glu_bwd.
 *   - Results are deterministic and batch invariant: every output byte depends only on
 *     its own element (BF16 entries) or its own 32- or 16-element block.
 */
#ifndef GLU_MX_H
#define GLU_MX_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum glu_status {
  GLU_OK = 0,
  GLU_ERR_NULL = 1,        /* a required pointer is NULL */
  GLU_ERR_SHAPE = 2,       /* negative extent, block divisibility violated, extent overflow */
  GLU_ERR_ALIGN = 3,       /* a base pointer is not 16-byte aligned */
  GLU_ERR_STRIDE = 4,      /* a row stride is too small or not a multiple of 8 elements */
  GLU_ERR_ARG = 5,         /* unknown enum/flag, or a pointer given for a disabled output */
  GLU_ERR_OVERLAP = 6,     /* an output overlaps an input or another output */
  GLU_ERR_UNSUPPORTED = 7, /* a well-formed combination this library does not implement */
  GLU_ERR_HIP = 8          /* the HIP runtime refused the launch */
} glu_status;

/* Activation (every entry point takes all four). */
enum { GLU_SWIGLU = 0, GLU_GEGLU_TANH = 1, GLU_GEGLU_ERF = 2, GLU_RELU2 = 3 };

/* Operand layout.
 *   GLU_SPLIT : gate and up are two [M, N] matrices sharing the row stride ld_in.  The
 *               concatenated [gate | up] matrix of [MX] API is GLU_SPLIT with
 *               up = gate + N and ld_in = 2N.
 *   GLU_PAIRED: one [M, 2N] matrix passed as `gate` (`up` must be NULL) whose column 2j is
 *               gate_j and column 2j+1 is up_j ([NV] Supported contract, weight layout). */
enum { GLU_SPLIT = 0, GLU_PAIRED = 1 };

/* MXFP8 flags: the directions (both = GLU_ROWWISE | GLU_COLWISE), optionally ORed with
 * GLU_SF_SWIZZLED, which writes both E8M0 scale matrices in the zero-padded 128x4 layout
 * described for GLU_SF_128x4 below (a [rows, nb] scale matrix then takes Rp*Cp bytes with
 * Rp = ceil(rows/128)*128 and Cp = ceil(nb/4)*4; see glu_mxfp8_sf_bytes).  No page fixes a
 * layout for MXFP8 scales; this is the GEMM-ready block-scale layout of [NV] Supported
 * contract, offered as an option. */
enum { GLU_ROWWISE = 1, GLU_COLWISE = 2, GLU_SF_SWIZZLED = 4 };

/* NVFP4 scale-factor layout.
 *   GLU_SF_ROWMAJOR: [M, H/16] bytes.
 *   GLU_SF_128x4   : the 128x4 tiled layout named in [NV] Supported contract (scales row).
 *                    Rows are padded to Rp = ceil(M/128)*128 and scale columns to
 *                    Cp = ceil((H/16)/4)*4; scale (r, c) lives at byte
 *                    ((r/128)*(Cp/4) + c/4)*512 + (r%32)*16 + ((r%128)/32)*4 + c%4,
 *                    and the library writes zero to every padding byte.  The buffer must
 *                    hold Rp*Cp bytes. */
enum { GLU_SF_ROWMAJOR = 0, GLU_SF_128x4 = 1 };

/* GEMM operand codes (glu_gemm*): MXFP8 (E4M3, one per byte) or MXFP4 (E2M1, two per byte). */
enum { GLU_FMT_E4M3 = 0, GLU_FMT_E2M1 = 1 };

/* ---- GLU forward, BF16 output ([MX] Summary; [GE] Summary; [H] Fixed numerical paths)
 * h[m, j] = bf16(act(g) * up_j), g = gate_j, computed in FP32 and rounded once to nearest
 * even.  h is [M, N] with row stride ld_h.
 * Strides: when the operands are contiguous (GLU_SPLIT with ld_in == N, or GLU_PAIRED with
 * ld_in == 2N, and ld_h == N) any N is accepted (ragged widths such as 8193, [GE] Testing
 * Done).  Otherwise ld_in and ld_h must be multiples of 8 (GLU_ERR_STRIDE).
 * ld_in >= N (split) or >= 2N (paired), ld_h >= N. */
glu_status glu_fwd(int act, int layout, int64_t M, int64_t N, const uint16_t* gate,
                   const uint16_t* up, int64_t ld_in, uint16_t* h, int64_t ld_h,
                   void* stream);

/* ---- GLU backward, BF16 output ([GE] Testing Done: forward, da and db; [MX] API)
 * da = bf16(dh * up * act'(gate)), db = bf16(dh * act(gate)); dh is [M, N] with stride
 * ld_dh.  GLU_SPLIT: da and db are two [M, N] matrices with row stride ld_out (for the
 * concatenated [dGate | dUp] result pass db = da + N, ld_out = 2N).  GLU_PAIRED: da is one
 * interleaved [M, 2N] matrix (column 2j = dGate_j, 2j+1 = dUp_j), db must be NULL.
 * In place: da == gate and db == up (split) or da == gate (paired) with ld_out == ld_in is
 * allowed; each element is read before it is overwritten by the same thread.
 * Strides as for glu_fwd, with ld_dh and ld_out in place of ld_h. */
glu_status glu_bwd(int act, int layout, int64_t M, int64_t N, const uint16_t* gate,
                   const uint16_t* up, int64_t ld_in, const uint16_t* dh, int64_t ld_dh,
                   uint16_t* da, uint16_t* db, int64_t ld_out, void* stream);

/* ---- Fused forward + MXFP8 ([MX] Summary, API, Numerics and tests)
 * Quantizes h = bf16(act(gate) * up) without writing h.  Per 32-element block: amax =
 * max|h|; scale byte e + 127 for the smallest e in [-127, 127] with 448 * 2^e >= amax
 * (RCEIL); codes = E4M3(h * 2^-e), nearest even.  A block holding NaN or Inf gets scale
 * 0xFF and codes 0x7F.
 *   rowwise (flags & GLU_ROWWISE): q_row [M, N] codes, s_row [M, N/32] scales.
 *   (With GLU_SF_SWIZZLED, s_row and s_col hold the same scales in the 128x4 layout.)
 *   colwise (flags & GLU_COLWISE): q_col [N, M] codes (row j holds column j of h, i.e.
 *                                  the column-major [M, N]), s_col [N, M/32] scales.
 * A disabled direction's two pointers must be NULL.  Needs N % 32 == 0, and M % 32 == 0
 * when colwise (GLU_ERR_SHAPE); ld_in % 8 == 0 and ld_in <= 2^24 (GLU_ERR_STRIDE).  Output
 * buffers are contiguous; each code output's rows are at most 2^24 bytes (rowwise N,
 * colwise M; GLU_ERR_SHAPE). */
glu_status glu_fwd_mxfp8(int act, int layout, int64_t M, int64_t N, const uint16_t* gate,
                         const uint16_t* up, int64_t ld_in, int flags, uint8_t* q_row,
                         uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, void* stream);

/* ---- Fused backward + MXFP8 ([MX] API: backward returns [dGate | dUp] quantized)
 * The quantized matrix is X = [da | db], [M, 2N] (X[:, j] = da_j, X[:, N + j] = db_j), with
 * da, db as in glu_bwd and never written.  q_row [M, 2N], s_row [M, 2N/32], q_col [2N, M],
 * s_col [2N, M/32].  Only GLU_SPLIT is implemented (GLU_PAIRED -> GLU_ERR_UNSUPPORTED).
 * Needs N % 32 == 0, M % 32 == 0 when colwise, rowwise 2N <= 2^24 and colwise M <= 2^24
 * (GLU_ERR_SHAPE); ld_in and ld_dh multiples of 8 and at most 2^24 (GLU_ERR_STRIDE). */
glu_status glu_bwd_mxfp8(int act, int layout, int64_t M, int64_t N, const uint16_t* gate,
                         const uint16_t* up, int64_t ld_in, const uint16_t* dh,
                         int64_t ld_dh, int flags, uint8_t* q_row, uint8_t* s_row,
                         uint8_t* q_col, uint8_t* s_col, void* stream);

/* ---- Fused forward + NVFP4, global scale 1 ([NV] Summary, Supported contract)
 * h = bf16(act(gate) * up) is [M, H] and never written.  Per 16-element block of a row:
 * scale S = E4M3(amax / 6), nearest even; codes E2M1(h / S), nearest even, saturating at
 * +-6; S == 0 gives signed-zero codes.  A block holding NaN or Inf gets scale 0x7F and
 * zero codes.  q is [M, H/2] bytes with element 2k in the low nibble of byte k; sf is
 * GLU_SF_ROWMAJOR [M, H/16] or GLU_SF_128x4 (see above).
 * Needs H % 16 == 0 and H <= 2^26 (GLU_ERR_SHAPE), ld_in % 8 == 0 (GLU_ERR_STRIDE). */
glu_status glu_fwd_nvfp4(int act, int layout, int64_t M, int64_t H, const uint16_t* gate,
                         const uint16_t* up, int64_t ld_in, uint8_t* q, uint8_t* sf,
                         int sf_layout, void* stream);

/* ---- Two-level NVFP4: a global scale from the tensor's amax.  [NV] Supported contract
 * fixes global scale 1; real recipes relax it, which no page defines.  By reading, every
 * step is one IEEE FP32 operation:
 *   s = 2688 / amax (448 * 6), capped at 2^100; s = 1 when amax is zero, negative, NaN or
 *       infinite;
 *   block scale code = E4M3(bamax * fl(s / 6)), nearest even, saturating at 448;
 *   codes = E2M1(x * fl(s / S)), S = the scale code's value (0 when S == 0), nearest even,
 *       saturating at 6; dequantized x ~ code * S / s.
 * A block holding NaN or Inf gets scale 0x7F and zero codes. */

/* Amax pass: *amax = the largest |h| over h = bf16(act(gate) * up), [M, N] (NaN when some h
 * is NaN, 0 for an empty matrix); h is never written.  amax is device memory (4-byte
 * aligned), written on `stream` by kernels (no host synchronization).  Operands as for
 * glu_fwd_nvfp4: N % 16 == 0 and N <= 2^26 (GLU_ERR_SHAPE), ld_in % 8 == 0 (GLU_ERR_STRIDE),
 * 16-byte aligned (GLU_ERR_ALIGN). */
glu_status glu_amax(int act, int layout, int64_t M, int64_t N, const uint16_t* gate,
                    const uint16_t* up, int64_t ld_in, float* amax, void* stream);

/* Fused forward + two-level NVFP4: as glu_fwd_nvfp4, with the global encode scale of the
 * FP32 value at device pointer amax (normally glu_amax's output on the same stream, or an
 * amax kept from an earlier step).  The scale s itself is not stored: the consumer derives
 * it from the same amax. */
glu_status glu_fwd_nvfp4_gs(int act, int layout, int64_t M, int64_t H, const uint16_t* gate,
                            const uint16_t* up, int64_t ld_in, const float* amax, uint8_t* q,
                            uint8_t* sf, int sf_layout, void* stream);

/* ---- Merged gate/up block-scaled GEMM with the GLU as its epilogue ([NV] Summary: the
 * fold follows the merged GEMM; [MX] Performance: the fused-w13 MoE composite under an MXFP8
 * recipe; [MX] API: a fused w13 projection packs [gate | up]).  The pre-activation is never
 * written.
 *   Y = X W^T with X [M, K] and W [2N, K] block-scaled along K: E8M0 scales xs [M, K/32] and
 *   ws [2N, K/32] (one per 32-element block), codes in format fmt:
 *     GLU_FMT_E4M3 (MXFP8): xq [M, K], wq [2N, K], one code per byte;
 *     GLU_FMT_E2M1 (MXFP4, the closest form of [NV] Supported contract's packed E2M1
 *       values that gfx950's block-scaled matrix instruction takes): xq [M, K/2],
 *       wq [2N, K/2], two codes per byte, element 2j in the low nibble of byte j.
 *   All row-major, K contiguous.  W's rows in w_layout:
 *     GLU_SPLIT:  W = [W_gate | W_up], gate output j in row j, up in row N + j;
 *     GLU_PAIRED: pairwise-interleaved gate/up rows gate0, up0, gate1, up1, ... ([NV]
 *       Supported contract, weight layout row), gate j in row 2j, up in row 2j + 1.
 *   h = bf16(act(Y_gate[:, j]) * Y_up[:, j]), Y accumulated in FP32 by the matrix cores.
 * E4M3: the matrix cores add the products of each 8-element K chunk in a 14-bit fixed-point
 * window anchored at the chunk's largest product (smaller bits are dropped), then add the
 * chunk sums into FP32 one at a time.  Y thus differs from the exact product sum by at most
 * sum over chunks of 2^-10 * (largest |x_k w_k| of the chunk), plus (K/8) * 2^-23 * sum |x_k w_k|.
 * E2M1: the products of each aligned 16-element K chunk share both scales and span at most
 * 2^8, so each chunk sum is exact; the chunk sums are added into FP32 one at a time, and Y
 * is within (K/16) * 2^-23 * sum |x_k w_k| of the exact sum.
 * Each row of h depends only on that row of X and on W, bit for bit.
 * Needs K > 0 with K % 128 == 0 (E4M3) or K % 256 == 0 (E2M1), N % 128 == 0
 * (GLU_ERR_SHAPE); every operand and output below 2^31 bytes (GLU_ERR_SHAPE); 16-byte
 * aligned pointers (GLU_ERR_ALIGN); an unknown act, fmt or w_layout is GLU_ERR_ARG. */
glu_status glu_gemm(int act, int fmt, int w_layout, int64_t M, int64_t N, int64_t K,
                    const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                    uint16_t* h, int64_t ld_h, void* stream);
/* The same h quantized MXFP8 rowwise (as glu_fwd_mxfp8): q_row [M, N], s_row [M, N/32]. */
glu_status glu_gemm_mxfp8(int act, int fmt, int w_layout, int64_t M, int64_t N, int64_t K,
                          const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                          const uint8_t* ws, uint8_t* q_row, uint8_t* s_row, void* stream);
/* The same h quantized NVFP4 with global scale 1, as glu_fwd_nvfp4 quantizes its output
 * ([NV] Summary: the merged GEMM's GeGLU result leaves as packed NVFP4 and scales for the
 * down projection): q [M, N/2] packed E2M1 (even column in the low nibble), sf E4M3 scales
 * of 16-column blocks in sf_layout (GLU_SF_ROWMAJOR [M, N/16], or GLU_SF_128x4 with rows
 * padded to 128 and zero padding; glu_nvfp4_sf_bytes(M, N, sf_layout) bytes).
 * Requirements and errors as glu_gemm; an unknown sf_layout is GLU_ERR_ARG. */
glu_status glu_gemm_nvfp4(int act, int fmt, int w_layout, int64_t M, int64_t N, int64_t K,
                          const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                          const uint8_t* ws, uint8_t* q, uint8_t* sf, int sf_layout,
                          void* stream);
/* The same NVFP4 output with two-level scaling (as glu_fwd_nvfp4_gs): the global encode scale
 * comes from the FP32 value at device pointer amax, which a GEMM epilogue cannot know before
 * h exists, so it is the caller's (an amax kept from an earlier step, i.e. delayed scaling, or
 * glu_amax of an h computed earlier).  amax: 4-byte aligned (GLU_ERR_ALIGN), not NULL
 * (GLU_ERR_NULL), not overlapping the outputs (GLU_ERR_OVERLAP).  Otherwise as glu_gemm_nvfp4. */
glu_status glu_gemm_nvfp4_gs(int act, int fmt, int w_layout, int64_t M, int64_t N, int64_t K,
                             const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                             const uint8_t* ws, const float* amax, uint8_t* q, uint8_t* sf,
                             int sf_layout, void* stream);
/* Test hook: the FP32 GEMM alone, formed exactly as the fused kernels form it: y [M, 2N]
 * holds Y_gate in columns 0..N-1 and Y_up in N..2N-1, whatever w_layout. */
glu_status glu_mx_gemm_f32(int fmt, int w_layout, int64_t M, int64_t N, int64_t K,
                           const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                           const uint8_t* ws, float* y, void* stream);

/* ---- Fused backward + NVFP4, global scale 1 (no page defines an NVFP4 backward: the
 * placement is glu_bwd_mxfp8's, [MX] API; the block arithmetic is glu_fwd_nvfp4's, [NV]
 * Supported contract).  The quantized matrix is X = [da | db], [M, 2N], with da, db as in
 * glu_bwd and never written; 16-element row blocks never straddle da and db.  q is
 * [M, N] bytes (2N codes per row, element 2k in the low nibble of byte k); sf is
 * GLU_SF_ROWMAJOR [M, 2N/16] or GLU_SF_128x4 over [M, 2N/16] (glu_nvfp4_sf_bytes(M, 2N)).
 * Only GLU_SPLIT is implemented (GLU_PAIRED -> GLU_ERR_UNSUPPORTED).  Needs N % 16 == 0
 * and N <= 2^26 (GLU_ERR_SHAPE); ld_in, ld_dh multiples of 8 with ld_dh >= N
 * (GLU_ERR_STRIDE). */
glu_status glu_bwd_nvfp4(int act, int layout, int64_t M, int64_t N, const uint16_t* gate,
                         const uint16_t* up, int64_t ld_in, const uint16_t* dh,
                         int64_t ld_dh, uint8_t* q, uint8_t* sf, int sf_layout,
                         void* stream);

/* ---- Quantizer test hooks: the same device quantizer code, fed FP32 values
 * x is an FP32 [M, N] matrix with row stride ld_x (a multiple of 4; at most 2^23 for the
 * MXFP8 hook, whose output pitches are bounded as for glu_fwd_mxfp8).  Outputs and rules
 * exactly as glu_fwd_mxfp8 / glu_fwd_nvfp4 with x in place of h (the NVFP4 hook also needs
 * H <= 2^26); every FP32 input is quantized exactly (no intermediate rounding). */
glu_status glu_quant_mxfp8_f32(int64_t M, int64_t N, const float* x, int64_t ld_x, int flags,
                               uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                               uint8_t* s_col, void* stream);
glu_status glu_quant_nvfp4_f32(int64_t M, int64_t H, const float* x, int64_t ld_x,
                               uint8_t* q, uint8_t* sf, int sf_layout, void* stream);

/* ---- Measurement hook: the streaming probe.  Moves n_vec 16-byte vectors from each of the
 * n_src sources (1..3) into each of the n_dst destinations (1..4; dst_bytes = 4, 8 or 16
 * bytes per vector) with non-temporal loads and stores, one vector per thread, consecutive
 * workgroups on consecutive addresses: the practical HBM ceiling for that mix of read and
 * write streams, beside which the fused kernels' rates are read (a fused MXFP8 forward
 * reads two BF16 streams and writes one byte per element: n_src = 2, dst_bytes = 8 per
 * 8-element vector).  With x the XOR of the sources' vectors (32-bit words x0..x3),
 * destination k receives per vector x with x0 + k in place of x0 (dst_bytes = 16), the words
 * (x0 ^ x2) + k, x1 ^ x3 (8), or the word (x0 ^ x1 ^ x2 ^ x3) + k (4).  src and dst are host
 * arrays of device pointers (16-byte aligned); destinations may not overlap the sources or
 * each other.  Errors: GLU_ERR_ARG (counts, dst_bytes), GLU_ERR_SHAPE (n_vec < 0 or above
 * 2^36), GLU_ERR_NULL, GLU_ERR_ALIGN, GLU_ERR_OVERLAP. */
glu_status glu_stream_probe(int n_src, const void* const* src, int n_dst, void* const* dst,
                            int64_t n_vec, int dst_bytes, void* stream);

/* ---- Host-only validation: the exact checks the entry point of the same name runs
 * before launching, with the same arguments minus the stream.  Never calls HIP and never
 * dereferences a pointer, so it runs on machines without a GPU. */
glu_status glu_check_fwd(int act, int layout, int64_t M, int64_t N, const uint16_t* gate,
                         const uint16_t* up, int64_t ld_in, uint16_t* h, int64_t ld_h);
glu_status glu_check_bwd(int act, int layout, int64_t M, int64_t N, const uint16_t* gate,
                         const uint16_t* up, int64_t ld_in, const uint16_t* dh,
                         int64_t ld_dh, uint16_t* da, uint16_t* db, int64_t ld_out);
glu_status glu_check_fwd_mxfp8(int act, int layout, int64_t M, int64_t N,
                               const uint16_t* gate, const uint16_t* up, int64_t ld_in,
                               int flags, uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                               uint8_t* s_col);
glu_status glu_check_bwd_mxfp8(int act, int layout, int64_t M, int64_t N,
                               const uint16_t* gate, const uint16_t* up, int64_t ld_in,
                               const uint16_t* dh, int64_t ld_dh, int flags,
                               uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                               uint8_t* s_col);
glu_status glu_check_fwd_nvfp4(int act, int layout, int64_t M, int64_t H,
                               const uint16_t* gate, const uint16_t* up, int64_t ld_in,
                               uint8_t* q, uint8_t* sf, int sf_layout);
glu_status glu_check_amax(int act, int layout, int64_t M, int64_t N, const uint16_t* gate,
                          const uint16_t* up, int64_t ld_in, float* amax);
glu_status glu_check_fwd_nvfp4_gs(int act, int layout, int64_t M, int64_t H,
                                  const uint16_t* gate, const uint16_t* up, int64_t ld_in,
                                  const float* amax, uint8_t* q, uint8_t* sf, int sf_layout);
glu_status glu_check_gemm(int act, int fmt, int w_layout, int64_t M, int64_t N, int64_t K,
                          const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                          const uint8_t* ws, uint16_t* h, int64_t ld_h);
glu_status glu_check_gemm_mxfp8(int act, int fmt, int w_layout, int64_t M, int64_t N, int64_t K,
                                const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                                const uint8_t* ws, uint8_t* q_row, uint8_t* s_row);
glu_status glu_check_gemm_nvfp4(int act, int fmt, int w_layout, int64_t M, int64_t N, int64_t K,
                                const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                                const uint8_t* ws, uint8_t* q, uint8_t* sf, int sf_layout);
glu_status glu_check_gemm_nvfp4_gs(int act, int fmt, int w_layout, int64_t M, int64_t N,
                                   int64_t K, const uint8_t* xq, const uint8_t* xs,
                                   const uint8_t* wq, const uint8_t* ws, const float* amax,
                                   uint8_t* q, uint8_t* sf, int sf_layout);
glu_status glu_check_mx_gemm_f32(int fmt, int w_layout, int64_t M, int64_t N, int64_t K,
                                 const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                                 const uint8_t* ws, float* y);
glu_status glu_check_bwd_nvfp4(int act, int layout, int64_t M, int64_t N,
                               const uint16_t* gate, const uint16_t* up, int64_t ld_in,
                               const uint16_t* dh, int64_t ld_dh, uint8_t* q, uint8_t* sf,
                               int sf_layout);
glu_status glu_check_quant_mxfp8_f32(int64_t M, int64_t N, const float* x, int64_t ld_x,
                                     int flags, uint8_t* q_row, uint8_t* s_row,
                                     uint8_t* q_col, uint8_t* s_col);
glu_status glu_check_quant_nvfp4_f32(int64_t M, int64_t H, const float* x, int64_t ld_x,
                                     uint8_t* q, uint8_t* sf, int sf_layout);
glu_status glu_check_stream_probe(int n_src, const void* const* src, int n_dst, void* const* dst,
                                  int64_t n_vec, int dst_bytes);

/* Bytes of the scale buffer glu_fwd_nvfp4 / glu_quant_nvfp4_f32 write for this layout
 * (M*H/16 row-major, Rp*Cp for 128x4), or -1 for bad arguments. */
int64_t glu_nvfp4_sf_bytes(int64_t M, int64_t H, int sf_layout);

/* Bytes of one MXFP8 scale buffer covering a quantized [rows, cols] matrix (cols % 32 == 0):
 * rows*cols/32 row-major (swizzled = 0) or Rp*Cp in the 128x4 layout (swizzled = 1), or -1
 * for bad arguments.  Rowwise scales: rows = M, cols = N (2N for the backward).  Colwise
 * scales: rows = N (2N), cols = M. */
int64_t glu_mxfp8_sf_bytes(int64_t rows, int64_t cols, int swizzled);

/* ==== Operators around the GLU =======================================================
 * The norms on both sides of a block, the linear products beside the gate/up projection, and
 * the routing of tokens to experts: what a feed-forward block needs next to act(gate) * up.
 * The conventions above hold.  Data is BF16 unless said otherwise, arithmetic FP32.  Entry
 * points that need scratch memory take `work` of at least *_work_bytes bytes (16-byte
 * aligned; its contents need not be kept).  Results are deterministic. */

/* ---- Block norms
 *   x' = res_scale x + gate * z,  z = N(y) w_post (GLU_NORM_POST) or z = y
 *   h  = N(x') w_pre + b_pre                      (GLU_NORM_PRE)
 *   N(v) = v / sqrt(mean(v^2) + eps)              (GLU_NORM_RMS)
 *        = (v - mean v) / sqrt(var v + eps)       (GLU_NORM_LAYER)
 * x, x' are [M, H] BF16, or FP32 with GLU_NORM_F32_STREAM; y, h are BF16 [M, H]; h is formed
 * from the unrounded x'.  gate, w_pre, b_pre, w_post are BF16, or FP32 with
 * GLU_NORM_F32_PARAMS; a NULL one is left out of the formula.  The first three are [H], or
 * with GLU_NORM_{GATE,W,B}_GROUPED [groups, H], one row per M / groups consecutive rows of x
 * (a request's adaptive scale, shift and gate; groups = M gives one per row).
 * y may be NULL (x' = x: no x_out, no gate, GLU_NORM_PRE only).  H <= 16384, any H and any
 * row stride >= H; M < 2^31.  stats is FP32 [M, 4], kept for the backward: the mean and the
 * reciprocal root of y's row, then of x's.
 * glu_block_norm_mxfp8 writes h as MXFP8 rowwise instead (codes q [M, H], scales s [M, H/32],
 * byte for byte the library's quantizer applied to the BF16 h): an operand of glu_gemm.
 * H % 32 == 0 and row strides of x, y and x_out multiples of 8. */
enum { GLU_NORM_RMS = 0, GLU_NORM_LAYER = 1 };
enum {
  GLU_NORM_PRE = 1, GLU_NORM_POST = 2, GLU_NORM_F32_STREAM = 4, GLU_NORM_F32_PARAMS = 8,
  GLU_NORM_GATE_GROUPED = 16, GLU_NORM_W_GROUPED = 32, GLU_NORM_B_GROUPED = 64
};
glu_status glu_block_norm(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x, int64_t ld_x,
                          const uint16_t* y, int64_t ld_y, const void* gate, const void* w_pre,
                          const void* b_pre, const void* w_post, float res_scale, float eps, void* x_out,
                          int64_t ld_xo, uint16_t* h, int64_t ld_h, float* stats, void* stream);
glu_status glu_block_norm_mxfp8(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                                int64_t ld_x, const uint16_t* y, int64_t ld_y, const void* gate,
                                const void* w_pre, const void* b_pre, const void* w_post, float res_scale,
                                float eps, void* x_out, int64_t ld_xo, uint8_t* q, uint8_t* s, float* stats,
                                void* stream);

/* Gradients of x' and h with respect to everything.  dx_out (the stream's type; NULL: zero)
 * and dh are the gradients of x' and h; dx has the stream's type, dy is BF16, and dgate,
 * dw_pre, db_pre, dw_post have the parameters' type and shape (NULL: not wanted).  x, y and
 * the parameters are the forward's.  With M == 0 the parameters' gradients are zero. */
int64_t glu_block_norm_bwd_work_bytes(int64_t M, int64_t H, int64_t groups);
glu_status glu_block_norm_bwd(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                              int64_t ld_x, const uint16_t* y, int64_t ld_y, const float* stats,
                              const void* dx_out, int64_t ld_dxo, const uint16_t* dh, int64_t ld_dh,
                              const void* gate, const void* w_pre, const void* w_post, float res_scale,
                              void* dx, int64_t ld_dx, uint16_t* dy, int64_t ld_dy, void* dgate, void* dw_pre,
                              void* db_pre, void* dw_post, void* work, int64_t work_bytes, void* stream);

/* ---- Linear products
 *   p = x W^T + b,  y = act(p) + residual
 * x [M, K], w [groups, N, K] contiguous, bias [groups, N] or NULL, residual [M, N] or NULL,
 * y [M, N], all BF16; sums, bias, activation and residual in FP32, rounded once.  pre, if not
 * NULL, receives p as FP16 [M, N] (clamped to the FP16 range) for the backward.
 * offsets NULL: one W for all rows (groups == 1).  Otherwise int32 [groups + 1] on the device,
 * non-decreasing, and rows offsets[e] .. offsets[e + 1] - 1 go through W and b number e; rows
 * outside every group give zero rows of y (and pre), without bias or residual.  Offsets
 * outside 0 .. M are taken as the nearer end.
 * N and K are multiples of 8 up to 2^20, row strides multiples of 8 up to 2^21, groups <= 1024.
 * glu_linear_work_bytes: grouped is 1 when offsets are given. */
enum { GLU_LINEAR_NONE = 0, GLU_LINEAR_SILU = 1, GLU_LINEAR_GELU = 2 /* tanh */, GLU_LINEAR_GELU_ERF = 3 };
int64_t glu_linear_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, int grouped);
glu_status glu_linear(int act, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                      const uint16_t* x, int64_t ld_x, const uint16_t* w, const uint16_t* bias,
                      const uint16_t* residual, int64_t ld_res, uint16_t* y, int64_t ld_y, uint16_t* pre,
                      void* work, int64_t work_bytes, void* stream);

/* dp = dy act'(p);  dx = dp W,  dw[e] = dp^T x and db[e] = sum of dp over the rows of group e.
 * pre is the forward's (NULL when act is GLU_LINEAR_NONE).  dx [M, K], dw [groups, N, K],
 * db [groups, N], BF16, each NULL when not wanted.  Rows outside every group give zero rows of dx.
 * The residual's gradient is dy itself, in rows outside every group zero. */
int64_t glu_linear_bwd_work_bytes(int act, int64_t M, int64_t N, int64_t K, int64_t groups, int grouped,
                                  int with_bias);
glu_status glu_linear_bwd(int act, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                          const uint16_t* dy, int64_t ld_dy, const uint16_t* x, int64_t ld_x, const uint16_t* w,
                          const uint16_t* pre, uint16_t* dx, int64_t ld_dx, uint16_t* dw, uint16_t* db,
                          void* work, int64_t work_bytes, void* stream);

/* ---- Expert routing
 * glu_moe_sort: rows[t, j] = the place of choice (t, j) when all choices are sorted by expert,
 * ties in reading order; -1 where ids[t, j] is no expert number (a dropped choice).  ids is
 * int32 or int64 (id_bytes 4 or 8) [tokens, choices], rows int32 of that shape, offsets int32
 * [experts + 1]: expert e has places offsets[e] .. offsets[e + 1] - 1.  experts <= 1024,
 * tokens * choices < 2^31.
 * glu_moe_permute: xs[rows[t, j]] = x[t], rows of row_bytes bytes of any type (strides in
 * bytes); rows of xs [tokens * choices] past offsets[experts] are written as zero.
 * glu_moe_combine: out[t] = residual[t] + sum over j of weights[t, j] y[rows[t, j]], dropped
 * choices left out; weights FP32, NULL for ones (then it is the gradient of permute).
 * glu_moe_combine_bwd: dy[rows[t, j]] = weights[t, j] dout[t], with the rows past
 * offsets[experts] zero, and dweights[t, j] = <dout[t], y[rows[t, j]]> (0 where dropped). */
int64_t glu_moe_sort_work_bytes(int64_t tokens, int64_t choices, int experts);
glu_status glu_moe_sort(int64_t tokens, int64_t choices, int experts, const void* ids, int id_bytes, int32_t* rows,
                        int32_t* offsets, void* work, int64_t work_bytes, void* stream);
glu_status glu_moe_permute(int64_t tokens, int64_t choices, int experts, int64_t row_bytes, const void* x,
                           int64_t ld_x, const int32_t* rows, const int32_t* offsets, void* xs, int64_t ld_xs,
                           void* stream);
glu_status glu_moe_combine(int64_t tokens, int64_t choices, int64_t H, const uint16_t* y, int64_t ld_y,
                           const int32_t* rows, const float* weights, const uint16_t* residual, int64_t ld_res,
                           uint16_t* out, int64_t ld_out, void* stream);
glu_status glu_moe_combine_bwd(int64_t tokens, int64_t choices, int64_t H, int experts, const uint16_t* dout,
                               int64_t ld_dout, const uint16_t* y, int64_t ld_y, const int32_t* rows,
                               const float* weights, const int32_t* offsets, uint16_t* dy, int64_t ld_dy,
                               float* dweights, void* stream);

/* Argument checks of the entry points above, as for the others. */
glu_status glu_check_block_norm(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                                int64_t ld_x, const uint16_t* y, int64_t ld_y, const void* gate,
                                const void* w_pre, const void* b_pre, const void* w_post, float res_scale,
                                float eps, void* x_out, int64_t ld_xo, uint16_t* h, int64_t ld_h, float* stats);
glu_status glu_check_block_norm_mxfp8(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                                      int64_t ld_x, const uint16_t* y, int64_t ld_y, const void* gate,
                                      const void* w_pre, const void* b_pre, const void* w_post, float res_scale,
                                      float eps, void* x_out, int64_t ld_xo, uint8_t* q, uint8_t* s, float* stats);
glu_status glu_check_block_norm_bwd(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                                    int64_t ld_x, const uint16_t* y, int64_t ld_y, const float* stats,
                                    const void* dx_out, int64_t ld_dxo, const uint16_t* dh, int64_t ld_dh,
                                    const void* gate, const void* w_pre, const void* w_post, float res_scale,
                                    void* dx, int64_t ld_dx, uint16_t* dy, int64_t ld_dy, void* dgate,
                                    void* dw_pre, void* db_pre, void* dw_post, void* work, int64_t work_bytes);
glu_status glu_check_linear(int act, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                            const uint16_t* x, int64_t ld_x, const uint16_t* w, const uint16_t* bias,
                            const uint16_t* residual, int64_t ld_res, uint16_t* y, int64_t ld_y, uint16_t* pre,
                            void* work, int64_t work_bytes);
glu_status glu_check_linear_bwd(int act, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                                const uint16_t* dy, int64_t ld_dy, const uint16_t* x, int64_t ld_x,
                                const uint16_t* w, const uint16_t* pre, uint16_t* dx, int64_t ld_dx,
                                uint16_t* dw, uint16_t* db, void* work, int64_t work_bytes);
glu_status glu_check_moe_sort(int64_t tokens, int64_t choices, int experts, const void* ids, int id_bytes,
                              int32_t* rows, int32_t* offsets, void* work, int64_t work_bytes);
glu_status glu_check_moe_permute(int64_t tokens, int64_t choices, int experts, int64_t row_bytes, const void* x,
                                 int64_t ld_x, const int32_t* rows, const int32_t* offsets, void* xs,
                                 int64_t ld_xs);
glu_status glu_check_moe_combine(int64_t tokens, int64_t choices, int64_t H, const uint16_t* y, int64_t ld_y,
                                 const int32_t* rows, const float* weights, const uint16_t* residual,
                                 int64_t ld_res, uint16_t* out, int64_t ld_out);
glu_status glu_check_moe_combine_bwd(int64_t tokens, int64_t choices, int64_t H, int experts, const uint16_t* dout,
                                     int64_t ld_dout, const uint16_t* y, int64_t ld_y, const int32_t* rows,
                                     const float* weights, const int32_t* offsets, uint16_t* dy, int64_t ld_dy,
                                     float* dweights);

/* Static text for a status code (never NULL). */
const char* glu_status_string(glu_status status);

/* Library version as major*10000 + minor*100 + patch. */
int glu_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GLU_MX_H */
