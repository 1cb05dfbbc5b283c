/*
 * qmm.h -- C ABI of the fused low-bit dequantize-matmul library for MI355X (gfx950).
 *
 * The operations follow three public pages:
 *   [P1] hip-ep pull request 1318, "bits=2 MatMulNBits" (2-bit phi4-14B): sections
 *        "Why" and "What", commit 1 -- MatMulNBits with per-block fp16 scales and
 *        a zero point that is a tensor or, when all equal, a scalar; a GEMV that
 *        reads fp32 A and writes fp32 C; prefill tiles that cast A to fp16 once.
 *   [P2] hip-ep pull request 1328, "fused QMoE decode picks tiling up front":
 *        sections "Summary", "Why", "What", "Notes for reviewers" -- the top-k MoE
 *        decode fc1 -> SwiGLU -> fc2 with an int8-activation variant, tiling chosen
 *        before the first call computes, HIP error state cleared on entry,
 *        num_experts argument, scratch-only timing, capture fallback.
 *   [P3] bitsandbytes pull request 1979, "[ROCm] Fused 4-bit SIMT GEMM":
 *        sections "Summary" and "Technical details" -- 16-entry codebook (NF4/FP4)
 *        4-bit weights with per-block absmax, decoded inside the GEMM; A must be
 *        contiguous row-major.
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library
 *     keeps no reference to them after the call returns.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Compute entry points only enqueue work on it and return without waiting,
 *     except the first call of a new shape, which times tiling candidates first
 *     (synchronizing the stream; never while the stream is being captured).
 *   - On entry the sticky HIP error state is cleared (hipGetLastError), so an
 *     error left by unrelated earlier work is not reported as this call's.
 *   - Return value (qmm_status): 0 on success; a negative QMM_E_* code if the
 *     arguments were refused before anything was launched; a positive value is
 *     the hipError_t reported after the launches.
 *   - Matrices are dense and row-major: A[M][K] (row stride K), C[M][N].
 *   - Packed weights: W[N][nblk][block*bits/8] bytes, nblk = ceil(K/block).
 *     Element k of row n lives in block b = k/block at position j = k%block, as
 *     the `bits`-wide field starting at bit j*bits of the block's little-endian
 *     bit stream (bit i of byte m is stream bit 8m + i; least significant field
 *     first, so a 3-bit field may continue into the next byte).  Codes of 2, 3 and
 *     4 bits are unsigned; 8-bit codes are signed bytes (two's complement). Codes
 *     past K in the last block are padding and are never read.
 *   - Dequantized weight (affine): w = fp32(fp32(q - zp) * fp32(scale)).
 *     Dequantized weight (codebook): w = fp32(codebook[q] * absmax).
 *   - Outputs are accumulated in fp32 and rounded once to the output dtype.
 *     Repeated calls with the same inputs give bit-identical outputs; the
 *     summation order depends only on (M-path, K, block, bits), never on the
 *     tiling chosen by the tuner.
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int qmm_status;

/* element types */
enum { QMM_F32 = 0, QMM_F16 = 1, QMM_BF16 = 2 };

/* zero-point kinds ([P1] "What", commit 1) */
enum {
  QMM_ZP_NONE = 0,     /* zp = 2^(bits-1) for every block (0 for signed 8-bit codes)  */
  QMM_ZP_PACKED = 1,   /* uint8 [N][ceil(nblk*bits/8)]: codes in W's field layout (signed
                          bytes for 8-bit weights)                                      */
  QMM_ZP_F16 = 2,      /* fp16 [N][nblk]                                              */
  QMM_ZP_UNIFORM = 3   /* the scalar `uniform_zp`; the zp pointer is never read       */
};

/* MoE decode modes ([P2] "Summary": fp decode and its dp4a variant) */
enum { QMOE_FP = 0, QMOE_INT8_ACT = 1 };

/* refusal codes (negative): nothing was launched */
enum {
  QMM_OK = 0,
  QMM_E_NULL = -1,       /* a required pointer is NULL                                  */
  QMM_E_DTYPE = -2,      /* unsupported element type                                    */
  QMM_E_BITS = -3,       /* bits not in {2, 3, 4, 8} (MoE: 4; activation ops: 8, 16)    */
  QMM_E_BLOCK = -4,      /* block not a power of two in [16, 256] (3-bit weights and
                            MoE: >= 32)                                                 */
  QMM_E_SHAPE = -5,      /* a size is negative or out of range                          */
  QMM_E_ALIGN = -6,      /* a pointer is not aligned as the kernels require             */
  QMM_E_WORKSPACE = -7,  /* workspace/scratch missing or smaller than the query says    */
  QMM_E_MODE = -8,       /* unknown zero-point kind or MoE mode                         */
  QMM_E_DEVICE = -9,     /* no usable gfx950 device / library not initialised           */
  QMM_E_PARAM = -10      /* a quantization scale not finite and positive, or a zero
                            point outside the code range                                */
};

/* ---------------------------------------------------------------------------
 * qmm_nbits -- C[M][N] = A[M][K] . dequant(W)^T (+ bias)       ([P1] "What", commit 1)
 *
 *   A        [M][K] of a_type (QMM_F32, QMM_F16, QMM_BF16), contiguous, 16-byte aligned.
 *   W        packed codes, bits in {2, 3, 4, 8} ([P1] kernel unit-test leaves Wu2, Wu3,
 *            Wu4, Wi8; 8 = signed), block in {16, 32, 64, 128, 256} (3 bits: >= 32).
 *   scales   fp16 [N][nblk].
 *   zp       per zp_kind (see above); uniform_zp used only for QMM_ZP_UNIFORM.
 *   bias     [N] of c_type, or NULL.
 *   C        [M][N] of c_type.
 *   workspace, workspace_bytes: device scratch of at least
 *            qmm_nbits_workspace_bytes(M, K, N, a_type) bytes (may be NULL when that is 0).
 * Paths: M <= 8 runs the weight-streaming GEMV, which reads A in its own type
 * and accumulates in fp32.  M > 8 runs a matrix-core path: A is rounded to fp16
 * once into the workspace (rows of K rounded up to a multiple of 64, padded with
 * zeros, for any a_type), each weight is dequantized exactly in fp32 and rounded
 * to fp16, and the products are accumulated in fp32 on the fp16 matrix cores.
 * For 8 < M <= 64 with block >= 32 a skinny kernel (16-row M tiles, each weight
 * loaded once) runs; otherwise 256 x 256 output tiles.  When either grid would
 * not fill the chip, the reduction over K is split into a number of parts fixed
 * by the shape; fp32 partial sums [parts][M][N] follow A in the workspace and are
 * added in part order by a second kernel.
 * ------------------------------------------------------------------------- */
qmm_status qmm_nbits(const void* A, int a_type, int64_t M, int64_t K, int64_t N,
                     const uint8_t* W, int bits, int block, const uint16_t* scales,
                     const void* zp, int zp_kind, float uniform_zp, const void* bias,
                     void* C, int c_type, void* workspace, size_t workspace_bytes,
                     void* stream);

size_t qmm_nbits_workspace_bytes(int64_t M, int64_t K, int64_t N, int a_type);

/* Host-only check of qmm_nbits arguments: returns the status qmm_nbits would
 * refuse with (or QMM_OK).  Never dereferences a pointer, needs no GPU. */
qmm_status qmm_validate_nbits(const void* A, int a_type, int64_t M, int64_t K, int64_t N,
                              const uint8_t* W, int bits, int block, const uint16_t* scales,
                              const void* zp, int zp_kind, const void* bias, const void* C,
                              int c_type, const void* workspace, size_t workspace_bytes);

/* ---------------------------------------------------------------------------
 * qmm_codebook4 -- C[M][N] = A . (codebook[q] * absmax)^T (+ bias)
 *                                     ([P3] "Summary", "Technical details")
 *   A        [M][K] of a_type (QMM_F16 or QMM_BF16; QMM_F32 also accepted).
 *   W        packed 4-bit codes [N][nblk][block/2], block in {16..256}, power of two.
 *   absmax   fp32 [N][nblk].
 *   codebook fp32 [16] (any values; NF4/FP4 tables are sorted in [-1, 1]).
 *   bias     [N] of c_type, or NULL.   C [M][N] of c_type.
 *   workspace, workspace_bytes: device scratch of at least
 *            qmm_codebook4_workspace_bytes(M, K, N, a_type) bytes (NULL when that is 0).
 *            That size is nonzero from M = 4 on (except M = 4 with N * K <= 2^24).
 *            It is needed for M > 8, and for 4 <= M <= 8 with a 16-bit c_type (the
 *            size does not depend on c_type).
 * Paths: M <= 8 weight-streaming GEMV (fp32 FMA, codebook staged in LDS), except
 * 4 <= M <= 8 with a QMM_F16 or QMM_BF16 output and block >= 32, which takes the
 * skinny kernel below (the GEMV's work grows with M, the skinny kernel's does not up
 * to 16 rows; the fp16 operand rounding is well below the 16-bit output's).  M = 4
 * with N * K <= 2^24 stays on the GEMV (its four-row form is the faster there); the
 * path is a function of the shape and output type only.
 * The matrix-core paths round A to fp16 once into the workspace (as for qmm_nbits)
 * and use weights fp16(fp32(codebook[q] * absmax)): the skinny kernel for M <= 64
 * with block >= 32, 256 x 256 tiles otherwise (as for qmm_nbits).
 * ------------------------------------------------------------------------- */
qmm_status qmm_codebook4(const void* A, int a_type, int64_t M, int64_t K, int64_t N,
                         const uint8_t* W, int block, const float* absmax,
                         const float* codebook, const void* bias, void* C, int c_type,
                         void* workspace, size_t workspace_bytes, void* stream);

size_t qmm_codebook4_workspace_bytes(int64_t M, int64_t K, int64_t N, int a_type);

qmm_status qmm_validate_codebook4(const void* A, int a_type, int64_t M, int64_t K, int64_t N,
                                  const uint8_t* W, int block, const float* absmax,
                                  const float* codebook, const void* bias, const void* C,
                                  int c_type, const void* workspace, size_t workspace_bytes);

/* ---------------------------------------------------------------------------
 * Nested (double-quantized) absmax for the codebook format ([P3] "Testing plan":
 * nested and non-nested absmax).  Block i (flat index n * nblk + b) stores an 8-bit
 * code into a 256-entry fp32 table; `group` consecutive blocks share one fp32 scale,
 * and one fp32 offset is added back:
 *   absmax_i = fp32(fp32(table[codes[i]] * scales[i / group]) + offset)
 * ------------------------------------------------------------------------- */
typedef struct {
  const uint8_t* codes;  /* uint8 [N][nblk] (device)                          */
  const float* table;    /* fp32 [256] (device)                               */
  const float* scales;   /* fp32 [ceil(N * nblk / group)] (device)            */
  float offset;
  int group;             /* blocks per scale, >= 1 (bitsandbytes uses 256)    */
} qmm_nested_absmax;

/* out[i] = absmax_i for i < count (fp32, device); `absmax` is a HOST pointer to the
 * descriptor.  Bit-exact with the definition above. */
qmm_status qmm_dequantize_absmax_nested(const qmm_nested_absmax* absmax, int64_t count, float* out,
                                        void* stream);

/* qmm_codebook4 with nested absmax: the absmax of the N * nblk blocks is decoded once
 * into the workspace (one small launch), then qmm_codebook4 runs on it, so results
 * are those of qmm_codebook4 on the decoded values.  workspace: at least
 * qmm_codebook4_nested_workspace_bytes(M, K, N, a_type, block) bytes, 256-byte
 * aligned (the decoded absmax first, then qmm_codebook4's workspace). */
qmm_status qmm_codebook4_nested(const void* A, int a_type, int64_t M, int64_t K, int64_t N,
                                const uint8_t* W, int block, const qmm_nested_absmax* absmax,
                                const float* codebook, const void* bias, void* C, int c_type,
                                void* workspace, size_t workspace_bytes, void* stream);
size_t qmm_codebook4_nested_workspace_bytes(int64_t M, int64_t K, int64_t N, int a_type, int block);

/* ---------------------------------------------------------------------------
 * qmm_fp16_uniform_value -- is every fp16 zero point bitwise equal?
 *                                     ([P1] "What", commit 1: detected once per buffer)
 *   zp       fp16 [count] (device).
 *   scratch  device buffer of at least qmm_uniform_scratch_bytes() bytes.
 *   is_uniform, value: HOST pointers receiving the flag and the fp32 value.
 * A NaN first element is never uniform; count == 0 is not uniform.
 * Synchronizes `stream` (call once per weight buffer, not per matmul).
 * ------------------------------------------------------------------------- */
qmm_status qmm_fp16_uniform_value(const uint16_t* zp, int64_t count, void* scratch,
                                  size_t scratch_bytes, int* is_uniform, float* value,
                                  void* stream);
size_t qmm_uniform_scratch_bytes(void);

/* ---------------------------------------------------------------------------
 * Dequantize to a dense matrix out[N][K] (out_type QMM_F32 or QMM_F16).
 * Bit-exact with the definitions above (fp16 output is the RNE rounding of the
 * fp32 weight, i.e. the operand the matrix-core paths use).
 * ------------------------------------------------------------------------- */
qmm_status qmm_dequantize_nbits(const uint8_t* W, int bits, int block, const uint16_t* scales,
                                const void* zp, int zp_kind, float uniform_zp, int64_t N,
                                int64_t K, void* out, int out_type, void* stream);

qmm_status qmm_dequantize_codebook4(const uint8_t* W, int block, const float* absmax,
                                    const float* codebook, int64_t N, int64_t K, void* out,
                                    int out_type, void* stream);

/* ---------------------------------------------------------------------------
 * qmoe_decode_fused -- top-k MoE decode with u4 expert weights.
 *                                     ([P2] "Summary", "Why", "What")
 * For token t in [0,T) and slot j in [0,k) with expert e = expert_ids[t][j]:
 *   [g ; u] = W1_e . x'_t + b1_e     (fc1: 2I outputs, g = rows [0,I), u = rows [I,2I))
 *   h       = fp16(g * sigmoid(g) * u)
 *   z       = W2_e . h' + b2_e       (fc2: H outputs)
 *   Y[t]    = fp16( sum over j = 0..k-1 in order of expert_w[t][j] * z )
 * QMOE_FP: x' = x, h' = h.  QMOE_INT8_ACT: x' and h' are symmetric int8 per 32
 * consecutive values (scale fp32(amax/127), codes rint(fp32(v*fp32(127/amax))))
 * and the products with (q - zp) are summed exactly in int32 per 32 values.
 *
 *   X          fp16 [T][H]            Y fp16 [T][H]
 *   expert_ids int32 [T][k], each in [0, E)  (an id outside is clamped into it on device)
 *   expert_w   fp32 [T][k]
 *   fc1.W      uint8 [E][2I][nblk(H)][block/2]   fc1.scales fp16 [E][2I][nblk(H)]
 *   fc1.zp     uint8 [E][2I][ceil(nblk(H)/2)] packed u4, or NULL (zp = 8)
 *   fc1.bias   fp16 [E][2I] or NULL
 *   fc2.*      the same with [E][H][..] over K = I
 *   bits       4.  block in {32, 64, 128, 256} (int8 mode additionally needs
 *              H % 32 == 0 and I % 32 == 0).
 *   scratch    device buffer of at least qmoe_decode_scratch_bytes(T, H, I, k, mode),
 *              256-byte aligned.  Layout (each region at a 256-byte boundary): the
 *              sync words of the single-launch form in the first 8448 bytes (the same
 *              place for every shape and mode): uint32 [0] top arrival count, [2] error
 *              flag, then in each of the next 32 256-byte slots an arrival sub-counter
 *              and a phase word; then fp16 h [T][k][I] at offset 8448, then in
 *              int8 mode int8 x codes [T][H], fp32 x scales [T][H/32], int8 h codes
 *              [T][k][I], fp32 h scales [T][k][I/32].  The sync words must be zero
 *              before the first call on a buffer (zero the whole buffer once, e.g.
 *              hipMemset); every call leaves the counters zero again and the phases
 *              equal, at 0 or 1.  The error flag is set, and left set, by a call whose wait inside
 *              the launch gave up after 1 s (its output is then invalid).  Calls that
 *              share a scratch buffer must not overlap.
 *   Launches   one launch of all of it by default: a grid that is resident all at
 *              once (its size is the kernel's occupancy times the compute units) runs
 *              its fc1 share, publishes h, waits for every work-group's h and streams
 *              its fc2 share (first loads issued before the wait; int8 mode: each
 *              work-group quantizes h itself).  The two-kernel form (fc1 + SwiGLU,
 *              then fc2 + combine; int8 mode adds the h quantizer between them) runs
 *              instead where the up-front timing finds it more than 5% faster, or
 *              where no single-launch plan fits.  The one-launch form
 *              needs the compute units to itself for that wait: a kernel on another
 *              stream that holds them for more than 1 s makes the wait give up (error
 *              flag above; the call's Y is then filled with fp16 NaN and
 *              qmoe_decode_status reports it).  Every form gives the same bits.
 *   E          num_experts: the first call of a shape times tiling candidates on
 *              other expert sets, writing only scratch.
 * ------------------------------------------------------------------------- */
typedef struct {
  const uint8_t* W;
  const uint16_t* scales;
  const uint8_t* zp;    /* packed u4 or NULL */
  const uint16_t* bias; /* fp16 or NULL */
} qmoe_weights;

qmm_status qmoe_decode_fused(const uint16_t* X, int64_t T, int64_t H, int64_t I, int64_t E,
                             int k, const int32_t* expert_ids, const float* expert_w,
                             qmoe_weights fc1, qmoe_weights fc2, int bits, int block,
                             int mode, uint16_t* Y, void* scratch, size_t scratch_bytes,
                             void* stream);

size_t qmoe_decode_scratch_bytes(int64_t T, int64_t H, int64_t I, int k, int mode);

/* ---------------------------------------------------------------------------
 * qmoe_ragged_mm -- the expert matmul of a multi-token MoE burst ([P1]/[P2] "Kernel Unit
 * Test Results": qmoe_ragged_mm, leaf Xfp16_Wu4_Yfp16; [P2] "Related issue or design":
 * T-token bursts through the QMoE layer).
 *   Rows of X are grouped by expert: expert e owns rows row_offsets[e] ..
 *   row_offsets[e+1] - 1 (row_offsets [E+1] int32 on the device, nondecreasing,
 *   row_offsets[0] = 0, row_offsets[E] = R; values are clamped into [0, R] on the
 *   device, and rows no expert owns are not written).  For each such row r
 *     Y[r] = fp16( X[r] . W16_e^T + bias_e )
 *   with W16_e = fp16 of the exact dequantized u4 weight (w = fp32(fp32(q - zp) * s),
 *   zp 8 when w.zp is NULL) and the products accumulated in fp32 on the fp16 matrix
 *   cores (the operand rounding of the matrix-core paths of qmm_nbits).
 *   X      fp16 [R][K], 16-byte aligned, K a multiple of 8.
 *   w      W [E][N][nblk][block/2], scales fp16 [E][N][nblk], zp packed u4
 *          [E][N][ceil(nblk/2)] or NULL, bias fp16 [E][N] or NULL.
 *   bits   4.  block: power of two in [32, 256].   Y fp16 [R][N].
 *   One launch; tiles of 16 to 64 rows of one expert per work-group.
 * ------------------------------------------------------------------------- */
qmm_status qmoe_ragged_mm(const uint16_t* X, int64_t R, int64_t K, int64_t N, int64_t E,
                          const int32_t* row_offsets, qmoe_weights w, int bits, int block,
                          uint16_t* Y, void* stream);

/* qmoe_decode_fused_noalloc -- qmoe_decode_fused for callers that cannot allocate
 * (code under stream capture, tight serving loops, harnesses that forbid hipMalloc).
 * Same arguments and results as qmoe_decode_fused, without scratch: the scratch is a
 * static device array of QMOE_NOALLOC_SCRATCH_BYTES inside the library, one per
 * device, held until the process ends.  A shape that needs more
 * (qmoe_decode_scratch_bytes) is refused with QMM_E_WORKSPACE.  The call never times
 * tiling candidates: it uses the choice an earlier qmoe_decode_fused call made for the
 * shape, else the default tiling, and so calls no allocating routine.  All calls on
 * one device share the array: calls that overlap on one device (other streams, other
 * threads) race and must not be made. */
#define QMOE_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
qmm_status qmoe_decode_fused_noalloc(const uint16_t* X, int64_t T, int64_t H, int64_t I, int64_t E,
                                     int k, const int32_t* expert_ids, const float* expert_w,
                                     qmoe_weights fc1, qmoe_weights fc2, int bits, int block, int mode,
                                     uint16_t* Y, void* stream);

/* qmoe_decode_status -- whether a single-launch qmoe_decode_fused call on this scratch
 * buffer gave up its wait ([P2] "What": a call must not report an error it did not
 * cause, nor hide one it did).  Reads the error word of the scratch layout above into
 * *timed_out (HOST pointer: 1 = some call gave up, its Y was filled with fp16 NaN;
 * 0 = none), then clears it.  T, H, I, k, mode: those of the calls made on the buffer.
 * Synchronizes `stream`.  Returns
 * QMM_E_NULL / QMM_E_WORKSPACE / QMM_E_ALIGN for a missing, short or misaligned buffer,
 * or the hipError_t of the copy. */
qmm_status qmoe_decode_status(void* scratch, size_t scratch_bytes, int64_t T, int64_t H, int64_t I,
                              int k, int mode, int* timed_out, void* stream);

qmm_status qmm_validate_qmoe(const uint16_t* X, int64_t T, int64_t H, int64_t I, int64_t E,
                             int k, const int32_t* expert_ids, const float* expert_w,
                             qmoe_weights fc1, qmoe_weights fc2, int bits, int block, int mode,
                             const uint16_t* Y, const void* scratch, size_t scratch_bytes);

/* ---------------------------------------------------------------------------
 * Activation quantize / dequantize and the fused quantized SwiGLU
 *                       ([P1] "Why": the per-layer chain Q(gate) -> qsigmoid -> 2x qmul ->
 *                        Q(up) -> DQ; "What", commit 4: fused Q -> DQ round trip and
 *                        fused quantized SwiGLU, each exactly equal to the unfused chain)
 *
 * Per-tensor parameters (scale, zero_point); codes are uint8 (bits = 8) or uint16
 * (bits = 16).  Element by element:
 *   Q(x)    = min(max(rint(fp32(x / scale)) + zero_point, 0), 2^bits - 1)
 *             (ties to even, the quotient correctly rounded; a NaN quotient gives 0)
 *   DQ(q)   = fp32((q - zero_point) * scale)
 *   sigmoid = the fp32 rounding of 1 / (1 + e^-v), evaluated in fp64
 * x, y: [n] of x_type / y_type (QMM_F32, QMM_F16, QMM_BF16; 16-bit outputs are the
 * nearest value of the fp32 result).  Device pointers, element-aligned; codes
 * 2-byte aligned for bits = 16.  scale must be finite and > 0, zero_point in
 * [0, 2^bits - 1] (else QMM_E_PARAM); bits other than 8 and 16 give QMM_E_BITS.
 * n = 0 launches nothing.  The fused ops give the bits of the unfused chain.
 * ------------------------------------------------------------------------- */
typedef struct {
  float scale;
  int32_t zero_point;
} qmm_qparams;

qmm_status qmm_quantize_linear(const void* x, int x_type, int64_t n, qmm_qparams q, int bits,
                               void* codes, void* stream);
qmm_status qmm_dequantize_linear(const void* codes, int64_t n, qmm_qparams q, int bits, void* y,
                                 int y_type, void* stream);
/* y = DQ(Q(x)), y of x_type: one launch, no code tensor. */
qmm_status qmm_fake_quantize(const void* x, int x_type, int64_t n, qmm_qparams q, int bits,
                             void* y, void* stream);
/* codes_out = Q(sigmoid(DQ(codes_in; in)); out). */
qmm_status qmm_qsigmoid(const void* codes_in, int64_t n, qmm_qparams in, qmm_qparams out, int bits,
                        void* codes_out, void* stream);
/* c = Q(fp32(DQ(a; qa) * DQ(b; qb)); qc). */
qmm_status qmm_qmul(const void* a, qmm_qparams qa, const void* b, qmm_qparams qb, int64_t n,
                    qmm_qparams qc, int bits, void* c, void* stream);
/* The quantized SwiGLU chain in one launch, y of x_type:
 *   g = Q(gate; q[0]);  t = qsigmoid(g -> q[1]);  m = qmul(g, t -> q[2]);
 *   u = Q(up; q[3]);    h = qmul(m, u -> q[4]);   y = DQ(h; q[4]).
 * q: HOST array of five parameter pairs (gate, sigmoid, silu, up, out). */
qmm_status qmm_qswiglu(const void* gate, const void* up, int x_type, int64_t n, int bits,
                       const qmm_qparams* q, void* y, void* stream);

/* ---------------------------------------------------------------------------
 * qmm_nbits_dgrad, qmm_codebook4_dgrad -- the input gradient of a frozen low-bit projection:
 *   dX[M][K] = dY[M][N] . dequant(W)
 *   with W, scales, zp / absmax, codebook as for qmm_nbits / qmm_codebook4 (the same buffers;
 *   nested absmax: decode it once with qmm_dequantize_absmax_nested).
 *   dY [M][N] of dy_type, dX [M][K] of dx_type (any of the three types).  W 4-byte aligned.
 *   M <= 2^24, 1 <= K, N <= 2^20.
 * Operands as on the forward matrix-core paths, for every M: dY is rounded to fp16 after one
 * exact power-of-two scale per row (fp16 dY that is 16-byte aligned with N a multiple of 8 is
 * read in place), each weight is dequantized exactly in fp32 and rounded to fp16, products are
 * accumulated in fp32, and the result is rounded once.  An fp32 dX is off by about 2e-4 of its
 * norm; weights below 6e-5 (fp16's subnormals) lose more.  The _f32 entries below round neither.
 * A contraction of few tiles is split; the sums are joined several loads at a time where M K is a
 * multiple of 4, one by one otherwise (M = 1, K = 1024 against 1023, N = 8192: 16 and 50 us).
 *   workspace: at least qmm_dgrad_workspace_bytes(M, K, N) bytes, 256-byte aligned.
 * ------------------------------------------------------------------------- */
qmm_status qmm_nbits_dgrad(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N,
                           const uint8_t* W, int bits, int block, const uint16_t* scales,
                           const void* zp, int zp_kind, float uniform_zp, void* dX, int dx_type,
                           void* workspace, size_t workspace_bytes, void* stream);
qmm_status qmm_codebook4_dgrad(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N,
                               const uint8_t* W, int block, const float* absmax,
                               const float* codebook, void* dX, int dx_type, void* workspace,
                               size_t workspace_bytes, void* stream);
size_t qmm_dgrad_workspace_bytes(int64_t M, int64_t K, int64_t N);

/* The same gradients with dY and the dequantized weights as they are: only the fp32 sums and dX are
 * rounded, as in the forward product with up to 8 rows (what of a value lies below 2^-133 is
 * dropped).  For fp32 dX (relative L2 <= 1e-5), for weights
 * that fp16 does not hold (below 6e-5 it loses their bits: small absmax or scales) and for gradients
 * of a wide range in one row.  Costs about twice the matrix work for codes of up to 4 bits with
 * integer zero points, three times it otherwise, twice that for fp16 dY and three times for fp32 dY;
 * bf16 dY that is 16-byte aligned with N a multiple of 8 is read in place.
 *   workspace: at least qmm_dgrad_f32_workspace_bytes(dy_type, M, K, N) bytes, 256-byte aligned. */
qmm_status qmm_nbits_dgrad_f32(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N,
                               const uint8_t* W, int bits, int block, const uint16_t* scales,
                               const void* zp, int zp_kind, float uniform_zp, void* dX, int dx_type,
                               void* workspace, size_t workspace_bytes, void* stream);
qmm_status qmm_codebook4_dgrad_f32(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N,
                                   const uint8_t* W, int block, const float* absmax,
                                   const float* codebook, void* dX, int dx_type, void* workspace,
                                   size_t workspace_bytes, void* stream);
size_t qmm_dgrad_f32_workspace_bytes(int dy_type, int64_t M, int64_t K, int64_t N);

/* Host-only checks of the arguments, as qmm_validate_nbits. */
qmm_status qmm_validate_nbits_dgrad(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N,
                                    const uint8_t* W, int bits, int block, const uint16_t* scales,
                                    const void* zp, int zp_kind, const void* dX, int dx_type,
                                    const void* workspace, size_t workspace_bytes);
qmm_status qmm_validate_codebook4_dgrad(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N,
                                        const uint8_t* W, int block, const float* absmax,
                                        const float* codebook, const void* dX, int dx_type,
                                        const void* workspace, size_t workspace_bytes);
qmm_status qmm_validate_nbits_dgrad_f32(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N,
                                        const uint8_t* W, int bits, int block, const uint16_t* scales,
                                        const void* zp, int zp_kind, const void* dX, int dx_type,
                                        const void* workspace, size_t workspace_bytes);
qmm_status qmm_validate_codebook4_dgrad_f32(const void* dY, int dy_type, int64_t M, int64_t K,
                                            int64_t N, const uint8_t* W, int block,
                                            const float* absmax, const float* codebook,
                                            const void* dX, int dx_type, const void* workspace,
                                            size_t workspace_bytes);

/* ---------------------------------------------------------------------------
 * qmoe_grouped_mm -- the ragged expert product of 16-bit weights, and its gradients (layers
 * kept in 16 bits next to the low-bit ones of qmoe_ragged_mm, and their training).
 *   Rows are grouped by expert as for qmoe_ragged_mm (row_offsets [E+1] int32 on the device;
 *   values are clamped into [0, R]).  For each row r of expert e
 *     Y[r]    = X[r] . W_e^T (+ bias_e)
 *     dX[r]   = dY[r] . W_e
 *     dW_e    = sum over the rows r of expert e of dY[r]^T X[r];  dbias_e = sum of dY[r]
 *   (zeros for an expert without rows; rows no expert owns are not written and their values
 *   reach no result), products exact, fp32 sums in an order that depends only on the sizes and
 *   offsets, each output rounded once.
 *   X [R][K], dY [R][N], W [E][N][K] of `type` (QMM_F16 or QMM_BF16).  bias [E][N] of y_type or
 *   NULL.  Y [R][N] of y_type, dX [R][K] of dx_type, dW [E][N][K] and dbias [E][N] of dw_type;
 *   of qmoe_grouped_mm_grad's outputs each may be NULL (not computed).
 *   R <= 2^24, 1 <= K, N <= 2^20, 1 <= E <= 65535.  Any sizes and element alignment are served;
 *   rows of 16-byte multiples from 16-byte aligned tensors take the direct copies into LDS, others
 *   go through registers, which do not overlap the arithmetic: 2 to 6 times slower.
 *   Tiles are chosen by the mean rows per expert and no contraction is split: few long experts among
 *   many, or one small expert alone, leave part of the chip idle.
 * ------------------------------------------------------------------------- */
qmm_status qmoe_grouped_mm(const void* X, int type, int64_t R, int64_t K, int64_t N, int64_t E,
                           const int32_t* row_offsets, const void* W, const void* bias, void* Y,
                           int y_type, void* stream);
qmm_status qmoe_grouped_mm_grad(const void* dY, const void* X, int type, int64_t R, int64_t K,
                                int64_t N, int64_t E, const int32_t* row_offsets, const void* W,
                                void* dX, int dx_type, void* dW, void* dbias, int dw_type,
                                void* stream);

/* Host-only checks of the arguments, as qmm_validate_nbits. */
qmm_status qmm_validate_grouped_mm(const void* X, int type, int64_t R, int64_t K, int64_t N,
                                   int64_t E, const int32_t* row_offsets, const void* W,
                                   const void* bias, const void* Y, int y_type);
qmm_status qmm_validate_grouped_mm_grad(const void* dY, const void* X, int type, int64_t R,
                                        int64_t K, int64_t N, int64_t E, const int32_t* row_offsets,
                                        const void* W, const void* dX, int dx_type, const void* dW,
                                        const void* dbias, int dw_type);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection, and their gradients.
 *
 * Row m of a batch belongs to a request with adapter a = ids[m] (an id outside [0, L):
 * none).  Next to any projection of this library, whose output is `base`:
 *   T[m] = A_a x_m                       fp32, products exact, fp32 sums
 *   Y[m] = base[m] + s_a * (B_a T[m])    rounded once to Y's type; Y[m] = base[m] for rows
 *                                        without an adapter
 * and the gradients, for dY:
 *   dT[m] = s_a * (B_a^T dy_m)           fp32
 *   dX[m] = base[m] + A_a^T dT[m]        base: the projection's own input gradient
 *   dA_a  = sum over its rows m of dT[m] x_m^T;  dB_a = s_a * sum over m of dy_m T[m]^T
 * (zeros for an adapter without rows).  T and dT are not rounded below fp32, whatever the range of
 * a row's ranks (what of a value lies below 2^-133 is dropped); infinities and NaN give what the
 * formulas give (where |T| >= 2^-86), in their own rows and adapters.
 *
 *   X [M][K], dY [M][N], A [L][r][K], B [L][N][r], all of `type` (QMM_F16 or QMM_BF16).
 *   ids   int32 [M] (device), in any order.   scale fp32 [L] (device) or NULL (1).
 *   base  [M][N] (qmm_lora_add) or [M][K] (qmm_lora_grad) of base_type, or NULL (0); may be
 *         the output itself when the types agree.
 *   T     fp32 [M][r].  qmm_lora_add writes it when given (rows without an adapter: zeros);
 *         qmm_lora_grad reads it, or computes it again from X when NULL.
 *   dX / dA / dB of qmm_lora_grad: each may be NULL (not computed).  dA [L][r][K] and dB
 *         [L][N][r] of g_type.
 *   M <= 2^24, 1 <= K, N <= 2^21, 1 <= r <= 512, 1 <= L <= 32768.  Any sizes and element
 *   alignment are served; 16-byte aligned tensors with K, N, r multiples of 8 are the fastest.
 *   Past 64 rows (in qmm_lora_grad always) the rows are sorted by L + 1 work-groups that each read all
 *   ids, whether an adapter has rows or not: 5 us for up to 100 adapters, 20 at 1024, 100 at 8192.
 *   workspace: at least the bytes of the query, 256-byte aligned.  Calls that share a
 *   workspace must not overlap.  The sums' order depends only on the shape and the ids.
 * ------------------------------------------------------------------------- */
typedef struct {
  const void* A;       /* [L][r][K] */
  const void* B;       /* [L][N][r] */
  const float* scale;  /* [L] or NULL */
} qmm_lora_weights;

qmm_status qmm_lora_add(const void* X, int type, int64_t M, int64_t K, int64_t N, int r, int64_t L,
                        const int32_t* ids, qmm_lora_weights w, const void* base, int base_type,
                        void* Y, int y_type, float* T, void* workspace, size_t workspace_bytes,
                        void* stream);
size_t qmm_lora_add_workspace_bytes(int64_t M, int64_t K, int64_t N, int r, int64_t L);

qmm_status qmm_lora_grad(const void* dY, const void* X, int type, int64_t M, int64_t K, int64_t N,
                         int r, int64_t L, const int32_t* ids, qmm_lora_weights w, const float* T,
                         const void* base, int base_type, void* dX, int dx_type, void* dA, void* dB,
                         int g_type, void* workspace, size_t workspace_bytes, void* stream);
size_t qmm_lora_grad_workspace_bytes(int64_t M, int64_t K, int64_t N, int r, int64_t L);

/* Host-only checks of the arguments, as qmm_validate_nbits. */
qmm_status qmm_validate_lora_add(const void* X, int type, int64_t M, int64_t K, int64_t N, int r,
                                 int64_t L, const int32_t* ids, qmm_lora_weights w, const void* base,
                                 int base_type, const void* Y, int y_type, const float* T,
                                 const void* workspace, size_t workspace_bytes);
qmm_status qmm_validate_lora_grad(const void* dY, const void* X, int type, int64_t M, int64_t K,
                                  int64_t N, int r, int64_t L, const int32_t* ids,
                                  qmm_lora_weights w, const float* T, const void* base, int base_type,
                                  const void* dX, int dx_type, const void* dA, const void* dB,
                                  int g_type, const void* workspace, size_t workspace_bytes);

/* ---------------------------------------------------------------------------
 * A key/value cache in 4 or 8 bits, and attention over it.
 *
 * The cache is a pool of pages; a slot is page_id * page + place.  A key (or value) of one token
 * and head is a row of D codes, unsigned `bits`-wide fields, least significant first; `group`
 * consecutive dimensions share a fp16 scale s and offset o, and code c stands for c * s + o (not
 * rounded; s of either sign, though the store writes none below 0).  Dimension d is the field at
 * position (d % W) * (D / W) + d / W of its row, W = 4 for keys and 16 for values: the order in which
 * the lanes of a matrix instruction take them.
 *   k, v                uint8 [pages][heads][page][D * bits / 8], 16-byte aligned
 *   k_params, v_params  fp16 [pages][heads][page][2][D / group] (scales, then offsets), 16-byte aligned
 *   bits in {4, 8}, D in {64, 128, 256}, group in {32, 64, 128} and <= D, page a power of two in
 *   [16, 65536], pages * page < 2^31, 1 <= heads <= 4096.
 * The descriptor is a HOST struct; its pointers are device pointers.
 *
 * qkv_cache_store -- quantizes the keys and values of T tokens into their slots.
 *   x = the value clamped to +-57344;  o = fp16(min of the group);  s = fp16(fp32(fp32(max - o) /
 *   (2^bits - 1))), at least 0;  c = the integer nearest to (x - o) / s as a real number, halves to the
 *   even one, clamped into the codes (0 when s is 0: a group whose steps would lie below 2^-25).
 *   A group that holds a NaN or an infinity reads back as NaN.
 *   K, V    [T][heads][D] of `type` (any of the three types), element (t, h, d) at
 *           t * row_stride + h * head_stride + d (strides in elements, >= 0).  Rows that are 16-byte
 *           aligned are the fastest.
 *   slots   int32 [T] (device), T <= 2^20.  A slot outside the pool: the token is not stored.  Of several
 *           tokens with one slot the last is stored; the search for them grows with T^2 and is what a call of
 *           more than 32768 tokens takes (several calls in order store the same, sooner).
 *
 * qkv_cache_load -- the values of T slots: K, V dense [T][heads][D] of `type`, fp32(c * s + o) rounded
 *   to it; zeros for a slot outside the pool.  K or V may be NULL (not read).  T <= 2^24.  In both calls
 *   T * heads <= 2^26.
 *
 * qkv_attention -- for query i of sequence b (n of them, the last n of its kv_len[b] tokens, so at
 * position p = kv_len[b] - n + i) and head a, over the tokens t of the sequence that it sees:
 *     S_t = scale * q . k_t;   out = sum_t e^(S_t) v_t / (sum_t e^(S_t) + e^(sinks[a]));
 *     lse = log(sum_t e^(S_t) + e^(sinks[a]))
 *   with head a reading cache head a / (q_heads / heads).  It sees t < kv_len[b] whose page is in the
 *   pool, with t <= p when causal, and t > p - window when window > 0 (causal only).  A query that sees
 *   nothing: out = 0, lse = the sink or -inf.  What hidden tokens hold, and what lies behind kv_len,
 *   reaches no result.
 *   Q       of `type` (QMM_F16 or QMM_BF16), element (row, a, d) at row * row_stride + a * head_stride
 *           + d (elements); T rows.  out dense [T][q_heads][D] of `type`; lse fp32 [T][q_heads] or NULL.
 *   cu_q    int32 [B + 1] (device): the queries of sequence b are the rows cu_q[b] .. cu_q[b + 1] - 1
 *           (clamped into [0, T], the first max_q of them); rows of no sequence are not written.
 *           NULL: row b is the one query of sequence b (T = B).
 *   kv_len  int32 [B] (device), clamped into [0, table_width * page].
 *   table   int32 [B][table_width] (device): pages of each sequence; one outside the pool is not seen.
 *   max_q   the greatest number of queries of a sequence (1 when cu_q is NULL); sets the grid.
 *   max_kv  the greatest kv_len expected (0: table_width * page, the most there can be): how the work is
 *           split depends on it, and the order of the sums; longer sequences are right all the same.
 *   sinks   fp32 [q_heads] (device) or NULL (none).  window 0: none.
 *   Codes enter the products as they are and scales are applied in fp32: S and lse carry fp32 sums'
 *   errors.  For the second product e^(S_t) s is rounded to fp16 (relative 2^-11; below 2^-20 of the largest
 *   e^(S_t) times the largest |s|, 2^-30 of that) for bf16 results and is held by two fp16 values (2^-22) for
 *   fp16 ones: so much of sum e^(S_t) |s| c, as codes are not centred; with many rows, groups of
 *   32 and bf16 results e^(S_t) and c * s + o are rounded to fp16 instead.  There a value beyond fp16's
 *   range (the store writes none) counts as NaN where a row sees it.
 *   Queries are scaled by a power of two per row to fp16: elements are rounded to multiples of 2^-31 of the
 *   row's largest one or finer (of 2^-124 in rows below 2^-93).  A query with a NaN or an infinity gives NaN, and
 *   so may one with elements, or scale times elements, past 2^100.
 *   B <= 65535, T <= 2^24, q_heads <= 4096 a multiple of heads with q_heads / heads <= 512, max_q *
 *   q_heads / heads < 2^31; QMM_E_SHAPE also where max_q, heads and B ask for 2^24 work-groups or more.
 *   workspace: at least qkv_attention_workspace_bytes (max_kv as in the call, table_width * page for 0; no
 *   workspace where that is 0), 256-byte aligned; calls that share one must not overlap.  The order of the
 *   sums depends on the sizes, max_q, max_kv, the window and the lengths only: equal calls give equal bits.
 * ------------------------------------------------------------------------- */
typedef struct {
  uint8_t* k;
  uint8_t* v;
  uint16_t* k_params;
  uint16_t* v_params;
  int64_t pages;
  int heads, page, D, bits, group;
} qkv_cache;

qmm_status qkv_cache_store(const void* K, int64_t k_row_stride, int64_t k_head_stride, const void* V,
                           int64_t v_row_stride, int64_t v_head_stride, int type, int64_t T,
                           const int32_t* slots, const qkv_cache* cache, void* stream);
qmm_status qkv_cache_load(const qkv_cache* cache, const int32_t* slots, int64_t T, void* K, void* V, int type,
                          void* stream);
qmm_status qkv_attention(const void* Q, int64_t row_stride, int64_t head_stride, int type, int64_t T,
                         int q_heads, int64_t B, const int32_t* cu_q, const int32_t* kv_len,
                         const int32_t* table, int64_t table_width, int64_t max_q, int64_t max_kv,
                         float scale, int causal, int64_t window, const float* sinks,
                         const qkv_cache* cache, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);
size_t qkv_attention_workspace_bytes(int64_t T, int q_heads, int heads, int D, int64_t B, int64_t max_q,
                                     int64_t max_kv, int64_t window);

/* Host-only checks of the arguments, as qmm_validate_nbits. */
qmm_status qmm_validate_kv_store(const void* K, int64_t k_row_stride, int64_t k_head_stride, const void* V,
                                 int64_t v_row_stride, int64_t v_head_stride, int type, int64_t T,
                                 const int32_t* slots, const qkv_cache* cache);
qmm_status qmm_validate_kv_load(const qkv_cache* cache, const int32_t* slots, int64_t T, const void* K,
                                const void* V, int type);
qmm_status qmm_validate_kv_attention(const void* Q, int64_t row_stride, int64_t head_stride, int type,
                                     int64_t T, int q_heads, int64_t B, const int32_t* cu_q,
                                     const int32_t* kv_len, const int32_t* table, int64_t table_width,
                                     int64_t max_q, int64_t max_kv, float scale, int causal,
                                     int64_t window, const float* sinks, const qkv_cache* cache,
                                     const void* out, const float* lse, const void* workspace,
                                     size_t workspace_bytes);

/* ---------------------------------------------------------------------------
 * Tuning control and introspection.
 * qmm_tuning_mode: 0 = time candidates on the first call of a shape (default),
 *   1 = never time, always use the default tiling, 2 = force candidate
 *   `forced_index` (for tests: every candidate must give identical bits).
 * qmm_tuned_choice: the candidate index chosen for the last call of the given
 *   entry (0 = qmm_nbits GEMV, 1 = qmm_codebook4 GEMV, 2 = qmoe fc1, 3 = qmoe fc2,
 *   4 = qmoe single-launch form, -1 when the last MoE call used two kernels), or -1
 *   if none; qmm_num_candidates gives the candidate count per entry.  Forced MoE
 *   indices below n(2) * n(3) pick the two-kernel form (fc1 = index % n(2),
 *   fc2 = index / n(2)); index n(2) * n(3) + c picks candidate c of entry 4.
 * qmm_clear_tuning forgets every cached choice.
 * ------------------------------------------------------------------------- */
qmm_status qmm_set_tuning(int mode, int forced_index);
int qmm_num_candidates(int entry);
int qmm_tuned_choice(int entry);
void qmm_clear_tuning(void);

/* GEMV candidates of entries 0 and 1: indices 0, 1, 2 are the v_dot8 / fp32 kernels
 * with 1, 2, 4 weight rows per lane; 3 is the matrix-core form of the 2-bit GEMV
 * (v_mfma_scale_f32_16x16x128_f8f6f4: the activation digit planes as e4m3 rows, the
 * codes as e2m1 nibbles, every product and sum exact; 16 weight rows per wave).  All
 * four give the same bits.  Where the matrix-core form does not serve a shape, index 3
 * runs the v_dot8 kernel with 2 rows per lane and the up-front timing skips it.
 * qmm_nbits_gemv_matrix_core_form: 1 when qmm_nbits at this shape (16-byte aligned
 * W, A and scales) has the matrix-core form among its candidates: bits = 2, M = 1,
 * block = 64 with ceil(K / 64) a multiple of 8, the activations' operand (4 KiB per
 * 256 codes) within LDS, and the lanes-per-row split of the v_dot8 kernel (fixed by K
 * and N) of 16 or 32 lanes, with ceil(K / 256) a multiple of a quarter of it; else 0. */
int qmm_nbits_gemv_matrix_core_form(int64_t M, int64_t K, int64_t N, int bits, int block);

/* The selection rule of the up-front timing, exposed for host-only checks:
 * times_us[r * ncand + c] is round r of candidate c; round 0 is discarded, the
 * least total over rounds 1..rounds-1 wins, ties go to the lower index.
 * Returns -1 for bad arguments. */
int qmm_tuner_pick(const double* times_us, int rounds, int ncand);

/* The MoE decode's choice between its single-launch forms and the two-kernel pair,
 * exposed for host-only checks: candidates 0 .. ncand-2 are single-launch forms and
 * candidate ncand-1 the pair, totals as in qmm_tuner_pick.  The fastest single launch
 * is chosen unless the pair's total is more than 5% below it (ties to the lower
 * index).  Returns -1 for bad arguments (ncand < 2 or rounds < 2). */
int qmm_tuner_pick_single_launch(const double* times_us, int rounds, int ncand);

/* ---------------------------------------------------------------------------
 * Measurement helper (not part of the computation): reads `bytes` of device memory
 * (16-byte aligned, a multiple of 16) once with 128-bit loads, `groups` work-groups of
 * 256 threads each reading one contiguous range, and writes the xor of what each
 * work-group read to sink[group] (uint32 [groups], device).  Timing it gives the HBM
 * read rate a plain streaming kernel reaches, the practical ceiling of the weight-
 * streaming kernels.  groups in [1, 2^20].
 * ------------------------------------------------------------------------- */
qmm_status qmm_hbm_read_probe(const void* buf, int64_t bytes, uint32_t* sink, int groups, void* stream);

/* Measurement helpers (not part of the computation): kernel execution times.
 * qmm_launch_timing_begin(n): from now on, the first n kernel launches that the library
 * makes from the calling host thread each record the start and the end of their execution
 * on the device (hipExtLaunchKernel with a pair of HIP events, created here on the current
 * device); the launches themselves are unchanged.  n in [1, 65536]; QMM_E_MODE if timing
 * is already on for this thread.  Do not switch it on around stream capture.
 * qmm_launch_timing_end(us, n_max, count): switches it off, waits for the recorded
 * launches, writes the duration in microseconds of each (launch order) to us[0..] (HOST
 * array, at most n_max values), the number of timed launches to *count (HOST), and frees
 * the events.  With timing off it writes *count = 0. */
qmm_status qmm_launch_timing_begin(int n);
qmm_status qmm_launch_timing_end(float* us, int n_max, int* count);

/* Human-readable name of a status code (static storage). */
const char* qmm_status_string(qmm_status s);

#ifdef __cplusplus
}
#endif
#endif /* QMM_H */
