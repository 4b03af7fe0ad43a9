/*
 * exl3.h -- C ABI of libexl3.so, the EXL3 trellis-quantized linear layer on sm_103a.
 *
 * The layer computes
 *
 *     y = svh * H_N( Wq^T-contraction( H_K(x * suh) * 2^-4 ) ) * 2^-3
 *
 * where H_K / H_N are block-diagonal 128-point Hadamard transforms and Wq is
 * decoded on the fly from 16x16 trellis tiles (cuda-exl3 README, "Why custom
 * kernels" and "One op per layer"; TensorFold PR #740, "Arithmetic").
 *
 * Conventions shared by every call:
 *  - All tensor pointers are DEVICE pointers owned by the caller, C-contiguous,
 *    16-byte aligned.  The library allocates nothing and keeps no per-layer
 *    state; it never synchronises the host.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Work is enqueued asynchronously on it.
 *  - Every argument is validated on the host before anything is launched.  An
 *    invalid call returns EXL3_EINVAL (or EXL3_EWORKSPACE) and launches nothing.
 *    A launch failure returns EXL3_ECUDA; exl3_last_error() gives the CUDA text.
 *  - fp16 / bf16 values are passed as their 16-bit patterns (uint16_t).
 *  - m == 0 is an empty batch: the call returns EXL3_OK and launches nothing;
 *    the activation, output and workspace pointers may then be NULL.
 *    m may be at most EXL3_MAX_ROWS.
 *  - k and n are multiples of 128 (whole Hadamard blocks; cuda-exl3 README,
 *    "Loading into a dim vLLM has padded").  bits is 1..8 (cuda-exl3 README,
 *    "What is supported").
 *  - Padded dims (same passage).  A dim padded for tensor parallelism is padded
 *    by whole 128-blocks, and the library needs nothing special for it:
 *      output (n) pad: the caller sets svh = 0 on the pad columns; those outputs
 *        are then exactly zero whatever trellis words sit behind them (every
 *        code decodes finite), and the real columns are unchanged because the
 *        output rotation mixes only inside a 128-column block;
 *      input (k) pad: when loading a checkpoint layer of K_real rows into a dim
 *        of K rows, the caller copies the K_real/16 trellis tile rows and the
 *        K_real suh entries per shard that exist and zeroes the rest (it must
 *        not read past the checkpoint's end), and the activations carry exact
 *        zeros on the pad positions (the producing layer's padded output
 *        already does).  The result equals the unpadded layer's, byte for byte
 *        for exl3_gemm (the extra k16 steps add exact zeros).
 */
#ifndef EXL3_H
#define EXL3_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { EXL3_CB_3INST = 0, EXL3_CB_MCG = 1, EXL3_CB_MUL1 = 2 } exl3_codebook_t;
typedef enum { EXL3_F16 = 0, EXL3_BF16 = 1 } exl3_dtype_t;
typedef enum {
  EXL3_OK = 0,
  EXL3_EINVAL = 1,       /* bad shape, pointer, alignment, width, codebook or shard map */
  EXL3_EUNSUPPORTED = 2, /* valid request this build does not implement */
  EXL3_EWORKSPACE = 3,   /* split-k accumulator too small */
  EXL3_ECUDA = 4         /* a CUDA launch or runtime call failed */
} exl3_status_t;

/* Largest batch (rows of x) one call accepts. */
#define EXL3_MAX_ROWS (1 << 22)

/* Maximum number of fused shards in one call (qkv = 3, gate_up = 2). */
#define EXL3_MAX_SHARDS 8

/*
 * exl3_input_transform -- input rotation of every shard in one pass over x.
 *
 * TensorFold PR #740, "Arithmetic" step 1; cuda-exl3 README, "One op per layer"
 * (activation transform fused, bf16 -> fp16 folded into the load).  For each
 * shard s, row r and 128-block b of k:
 *     xh[s][r][128b+i] = fp16_rne( 2^-4 * sum_j H[i][j] * (x[r][128b+j] * suh[s][128b+j]) )
 * with H[i][j] = (-1)^popcount(i & j), the product x*suh exact in fp32 and the
 * sum taken as a radix-2 butterfly in fp32 with a fixed order of adds.
 *
 *   x        device, [m][k] of x_dtype (bf16 or fp16)
 *   suh      device, fp16 [num_shards][k]
 *   xh       device, fp16 [num_shards][m][k] (output)
 */
exl3_status_t exl3_input_transform(const void* x, exl3_dtype_t x_dtype, int64_t m, int64_t k,
                                   const uint16_t* suh, int32_t num_shards, uint16_t* xh,
                                   void* stream);

/*
 * exl3_input_transform_swiglu -- the down-projection's input transform with the
 * gated MLP's SwiGLU folded in (cuda-exl3 README, "MoE throughput": folding
 * SwiGLU into the down-projection's input transform removes an elementwise
 * pass).  The pages print no formula; this library reads it as the usual
 * SwiGLU with the gate first:
 *     h[r][j]      = silu(g) * u,  g = gate_up[r][j], u = gate_up[r][k + j],
 *                    silu(g) = g / (1 + e^-g), in fp32
 *     xh[s][r][:]  = as exl3_input_transform with h in place of x
 * (the layout a gate_up layer fused as two shards of width k writes).
 *   gate_up  device, [m][2k] of dtype (bf16 or fp16), 16-byte aligned
 *   suh      device, fp16 [num_shards][k]
 *   xh       device, fp16 [num_shards][m][k] (output)
 * Validation and the empty batch as for exl3_input_transform.
 */
exl3_status_t exl3_input_transform_swiglu(const void* gate_up, exl3_dtype_t dtype, int64_t m, int64_t k,
                                          const uint16_t* suh, int32_t num_shards, uint16_t* xh,
                                          void* stream);

/*
 * exl3_gemm -- trellis decode fused into the contraction, output rotation fused
 * into the epilogue, all shards of a fused layer in one launch.
 *
 * cuda-exl3 README, "Why custom kernels" (a block owns its columns and the whole
 * k extent, so the output Hadamard and svh fold into the epilogue) and "Notes on
 * the format" (trellis and svh concatenate along n; one suh row, hence one xh
 * slice, per shard).  TensorFold PR #740, "Arithmetic" steps 2-3.
 *     z[r][c]  = sum_k xh[s(c)][r][k] * Wq[k][c]      (fp16 products, fp32 sums)
 *     y[r][c]  = out_rne( svh[c] * 2^-3 * sum_j H[i][j] z[r][128b+j] ),  c = 128b+i
 * Wq[k][c] is decoded from trellis tile (k/16, c/16).  The fp32 sum over k runs
 * in a fixed order that does not depend on m, so each row's bytes are the same
 * at every batch size.
 *
 *   xh         device, fp16 [num_shards][m][k] (exl3_input_transform's output)
 *   trellis    device, int16 [k/16][n/16][16*bits]
 *   bits       1..8;  cb: codebook id
 *   svh        device, fp16 [n]
 *   shard_cols HOST, int32 [num_shards+1]: 0 = c_0 < c_1 < ... < c_S = n, multiples
 *              of 128; shard s owns output columns [c_s, c_{s+1})
 *   y          device, [m][n] of y_dtype (output)
 *
 * Launch overlap: the GEMM kernel is launched with programmatic stream
 * serialization, and exl3_input_transform's kernel lets its dependents start
 * early.  So the GEMM may begin (and read trellis and svh) while the kernel
 * before it in the stream is still running, provided that kernel allows it;
 * it reads xh and writes y only after that kernel has completed.  A caller's
 * own kernel that allows early dependents must therefore not write the
 * trellis or svh that the following GEMM uses.
 */
exl3_status_t exl3_gemm(const uint16_t* xh, int64_t m, int64_t k, const int16_t* trellis,
                        int32_t bits, exl3_codebook_t cb, const uint16_t* svh,
                        const int32_t* shard_cols, int32_t num_shards, void* y,
                        exl3_dtype_t y_dtype, int64_t n, void* stream);

/*
 * Split-k variant.  cuda-exl3 README, "One op per layer" (split-k for narrow
 * layers: partials go to an fp32 accumulator that a second kernel turns into
 * outputs while zeroing it again); TensorFold PR #740, "Arithmetic" (k
 * blocks split into a number of parts fixed by the shape, parts added in part
 * order).  Part p covers a contiguous range of k: whole 256-row units when
 * k/128 is even and P <= k/256 (so a part never splits a four-atom stage),
 * else whole 128-row blocks, in either case part p takes units
 * [p*U/P, (p+1)*U/P) of the U units; its
 * fp32 partial goes to acc[p][r][c]; the epilogue sums p = 0..P-1 in order,
 * applies the output rotation, writes y and writes zeros back to acc.
 *
 * exl3_splitk_parts(k, n) is the number of parts P; it depends on the shape only
 * (never on m), so rows stay byte-equal across batch sizes.  It is a pure host
 * function.  exl3_splitk_workspace_bytes(m, k, n) = P * m * n * 4.
 *
 *   acc        device, fp32 [P][m][n].  Its contents on entry do not matter:
 *              each part stores every partial it owns (plain stores, no
 *              accumulation into acc) before the epilogue reads it.  The
 *              epilogue writes zeros back, the pages' re-zeroed accumulator,
 *              so with P > 1 acc is all zero when the call's work completes;
 *              nothing relies on that.  With P = 1 the call computes what
 *              exl3_gemm computes, with no partials and no epilogue, and
 *              leaves acc as it found it.  Calls that share one acc must be
 *              ordered on one stream.
 *   acc_bytes  size of acc in bytes; smaller than the workspace size -> EXL3_EWORKSPACE
 *   other arguments as exl3_gemm.
 * If a kernel of the call gives up on a bounded wait (exl3_device_status then
 * reports it), its part skips its stores and y is undefined for that call.
 */
int32_t exl3_splitk_parts(int64_t k, int64_t n);
size_t exl3_splitk_workspace_bytes(int64_t m, int64_t k, int64_t n);
exl3_status_t exl3_gemm_splitk(const uint16_t* xh, int64_t m, int64_t k, const int16_t* trellis,
                               int32_t bits, exl3_codebook_t cb, const uint16_t* svh,
                               const int32_t* shard_cols, int32_t num_shards, void* y,
                               exl3_dtype_t y_dtype, int64_t n, float* acc, size_t acc_bytes,
                               void* stream);

/*
 * Mixture of experts (cuda-exl3 README, "What is supported" and "MoE notes").
 * Routed (token, expert) pairs arrive block-aligned, the layout vLLM's
 * moe_align_block_size writes: pairs sorted by expert, each expert's run padded
 * to whole blocks of `block` rows, so every block belongs to one expert.
 *   sorted_ids    device int32 [rows]: pair index token * topk + slot of each
 *                 padded row; any value outside [0, num_tokens * topk) marks
 *                 a padding row
 *   block_expert  device int32 [rows / block]: expert of each block; -1 (or an
 *                 id >= num_experts) marks a block of no expert, which both
 *                 calls skip (such blocks may sit between live ones)
 *   block         16, 32 or 128; rows a multiple of block (16 is the pages'
 *                 floor, used when few tokens reach each expert: cuda-exl3
 *                 README, "MoE notes")
 *
 * exl3_moe_input_transform: since suh is per expert (and per shard), the input
 * rotation happens after routing: each padded row of a live block gets its
 * token's x rotated with its block's expert's suh, as exl3_input_transform
 * computes it; padding rows get zeros; rows of skipped blocks are not written.
 *   x    device, [num_tokens][k] of x_dtype
 *   suh  device, fp16 [num_experts][num_shards][k]
 *   xh   device, fp16 [num_shards][rows][k] (output)
 *
 * exl3_moe_gemm: the grouped GEMM.  Each live block's rows go through its
 * expert's layer exactly as exl3_gemm computes it (same fixed fp32 order, so a
 * row's bytes equal exl3_gemm's with that expert); skipped blocks' rows of y
 * are not written.
 *   xh       device, fp16 [num_shards][rows][k] (exl3_moe_input_transform's output)
 *   trellis  device, int16 [num_experts][k/16][n/16][16*bits] (experts stacked)
 *   svh      device, fp16 [num_experts][n]
 *   y        device, [rows][n] of y_dtype (output, in padded-row order; the
 *            weighted combine over each token's top-k rows is the caller's)
 * Validation and empty input as for exl3_gemm; EXL3_EINVAL also for a block
 * size other than 16, 32 or 128, rows not a multiple of it, or no experts.  The
 * kernel reads block_expert before it waits for the previous kernel in the
 * stream, like the trellis (see exl3_gemm).
 */
exl3_status_t exl3_moe_input_transform(const void* x, exl3_dtype_t x_dtype, int64_t num_tokens, int64_t k,
                                       const int32_t* sorted_ids, int64_t rows, int32_t topk,
                                       const int32_t* block_expert, int32_t block, const uint16_t* suh,
                                       int32_t num_shards, int32_t num_experts, uint16_t* xh, void* stream);
exl3_status_t exl3_moe_gemm(const uint16_t* xh, int64_t rows, int64_t k, const int16_t* trellis,
                            int32_t bits, exl3_codebook_t cb, const uint16_t* svh,
                            const int32_t* shard_cols, int32_t num_shards, const int32_t* block_expert,
                            int32_t block, int32_t num_experts, void* y, exl3_dtype_t y_dtype, int64_t n,
                            void* stream);

/*
 * exl3_moe_combine: the weighted sum of each token's top-k expert rows, the
 * step after the grouped GEMM (the pages leave it to the caller: cuda-exl3
 * README, "MoE notes"; the routing layout is the one above).
 *   out[t, :] = sum over s = 0 .. topk-1, in that order, of
 *               weights[t, s] * y[row(t, s), :]
 * where row(t, s) is the padded row of a live block (expert id in
 * [0, num_experts)) whose sorted_ids entry is the pair t * topk + s; a pair
 * with no such row adds nothing (a token with none gets zeros).  The sum is
 * fp32, one fused multiply-add per slot in slot order, then one rounding to
 * out_dtype; padding rows and rows of blocks of no expert are never read.
 *   y          device, [rows][n] of y_dtype (exl3_moe_gemm's output)
 *   weights    device, fp32 [num_tokens][topk] (the router's top-k weights)
 *   pair_rows  device, int32 [num_tokens * topk] scratch owned by the caller:
 *              the call writes the row of every routed pair into it first and
 *              checks each entry it reads against sorted_ids and block_expert,
 *              so it needs no clearing between calls
 *   out        device, [num_tokens][n] of out_dtype (output)
 * Each pair must appear in at most one row of a live block (the layout above
 * guarantees it; with duplicates the row taken is unspecified).  Two kernel
 * launches on `stream`, no synchronisation, no allocation.  EXL3_EINVAL for
 * sizes out of range, rows not a multiple of block, a block size other than
 * 16, 32 or 128, topk outside 1..64, no experts, or a missing or misaligned
 * pointer; num_tokens == 0 does nothing.
 */
exl3_status_t exl3_moe_combine(const void* y, exl3_dtype_t y_dtype, int64_t rows, int64_t n,
                               const int32_t* sorted_ids, const int32_t* block_expert, int32_t block,
                               int32_t num_experts, const float* weights, int64_t num_tokens, int32_t topk,
                               int32_t* pair_rows, void* out, exl3_dtype_t out_dtype, void* stream);

/*
 * Attention around the quantised layers: rotary positions, a paged key / value
 * cache in 16, 8 or 4 bits, attention over whole prompts and over the cache.
 * The pages have no counterpart to these calls: their layers run inside an
 * engine that brings its own.  Arithmetic, layouts and limits are this
 * library's own and are stated here.
 *
 * Heads of packed tokens are described by exl3_heads_t: element (t, h, d) at
 * data[t * token_stride + h * head_stride + d], strides in elements, positive
 * multiples of 8, data 16-byte aligned (so a call reads the heads it wants
 * straight from a fused projection's output).  head_dim is 64 or 128 (others:
 * EXL3_EUNSUPPORTED).  q_heads is a multiple of kv_heads; query head h uses key
 * head h / (q_heads / kv_heads).
 */
typedef struct {
  const void* data;
  int64_t token_stride, head_stride;
} exl3_heads_t;

/*
 * Rotary positions.  Pair i of a head turns by the angle position * f_i:
 *     (a, b) -> amplitude * (a cos - b sin, b cos + a sin)
 * The pairs are (x[i], x[i + rot_dim/2]) for EXL3_ROPE_HALF and
 * (x[2i], x[2i + 1]) for EXL3_ROPE_INTERLEAVED, i < rot_dim / 2; values from
 * rot_dim on stay.  f_i is given as a phase: turns per position in units of
 * 2^-64 (f_i / 2 pi * 2^64), so that position * phase modulo 2^64 is the exact
 * angle at every 32-bit position; its upper 32 bits, signed, times pi / 2^31 are
 * the angle in fp32.  Products and sums are fp32, rounded one by one, then once
 * to the type.
 *   phases     device, uint64 [rot_dim / 2]
 *   positions  device, int32 [tokens]
 *   rot_dim    multiple of 16, at most head_dim
 */
typedef enum { EXL3_ROPE_HALF = 0, EXL3_ROPE_INTERLEAVED = 1 } exl3_rope_layout_t;
typedef struct {
  const uint64_t* phases;
  const int32_t* positions;
  int32_t rot_dim;
  exl3_rope_layout_t layout;
  float amplitude;
} exl3_rope_t;

/*
 * exl3_rope_phases -- phases and amplitude of the usual frequencies
 * f_i = base^(-2i / rot_dim), scaled for long contexts (pure host function, 64
 * bits):
 *   EXL3_ROPE_PLAIN   f_i, amplitude 1
 *   EXL3_ROPE_LINEAR  f_i / factor, amplitude 1
 *   EXL3_ROPE_NTK     base * factor^(rot_dim / (rot_dim - 2)) in place of base, amplitude 1
 *   EXL3_ROPE_YARN    r_i = original_len * f_i / 2 pi turns over the original
 *                     context; g_i = clamp((r_i - slow) / (fast - slow), 0, 1);
 *                     f_i * (g_i + (1 - g_i) / factor), amplitude 0.1 ln(factor) + 1
 *                     (Peng et al., "YaRN: Efficient Context Window Extension of
 *                     Large Language Models").  The ramp is the paper's, over turns;
 *                     a checkpoint whose code ramps over the index i between two
 *                     rounded bounds has other frequencies there, and takes phases
 *                     of its own: any uint64 [rot_dim / 2] will do
 * factor >= 1, base > 1; fast > slow > 0 and original_len > 0 are read for YARN only.
 *   phases  HOST, uint64 [rot_dim / 2] (output);  amplitude  HOST (output)
 */
typedef enum { EXL3_ROPE_PLAIN = 0, EXL3_ROPE_LINEAR = 1, EXL3_ROPE_NTK = 2, EXL3_ROPE_YARN = 3 } exl3_rope_scaling_t;
exl3_status_t exl3_rope_phases(int32_t rot_dim, double base, exl3_rope_scaling_t scaling, double factor,
                               double fast, double slow, double original_len, uint64_t* phases,
                               float* amplitude);

/*
 * exl3_rope -- rotate `heads` heads of every token.  out may be x itself (same
 * strides): in place.  Out-of-place, out may not overlap x.
 *   out  device, strides as for exl3_heads_t
 */
exl3_status_t exl3_rope(const exl3_heads_t* x, exl3_dtype_t dtype, int64_t tokens, int32_t heads,
                        int32_t head_dim, const exl3_rope_t* rope, void* out, int64_t out_token_stride,
                        int64_t out_head_stride, void* stream);

/*
 * exl3_norm_rope -- the same with each head first divided by its root mean
 * square and multiplied by weights, and with positions of several axes:
 *     y[d] = x[d] * 1 / sqrt(sum_j x[j]^2 / head_dim + eps) * weight[d],  then rotated,
 * all in fp32, rounded to the type once, at the end.  (Squares are fp32: a head with values above 2^60 or so
 * comes out as zeros, one with a value that is not finite as NaN or zeros.)
 *   norm  NULL: none.  weight: device, 16-byte aligned, of `dtype`: row h, head_stride elements (a multiple of 8)
 *         from the one before, belongs to head h; head_stride 0: one row for all.  eps: a normal positive number
 *   rope  NULL (with a norm): nothing is rotated
 *   axes  NULL: positions [tokens] as for exl3_rope.  Else positions is [num_axes][tokens] and pair i turns by
 *         row axes[i] of it (time, height, width: any assignment of pairs to axes); axes: device, uint8
 *         [rot_dim / 2], an entry past the last axis is taken as the last
 * Other arguments as for exl3_rope; out may be x itself.
 */
typedef struct {
  const void* weight;
  int64_t head_stride;
  float eps;
} exl3_head_norm_t;
typedef struct {
  const uint8_t* axes;
  int32_t num_axes; /* 1 to 255 */
} exl3_rope_axes_t;
exl3_status_t exl3_norm_rope(const exl3_heads_t* x, exl3_dtype_t dtype, int64_t tokens, int32_t heads,
                             int32_t head_dim, const exl3_head_norm_t* norm, const exl3_rope_t* rope,
                             const exl3_rope_axes_t* axes, void* out, int64_t out_token_stride,
                             int64_t out_head_stride, void* stream);

/*
 * The paged cache.  Slot s is row s % page_size of page s / page_size.
 *   k, v              device, [num_pages][kv_heads][page_size][row bytes]
 *   k_scale, v_scale  device, bf16 [num_pages][kv_heads][page_size]; NULL for the 16-bit formats
 *   page_size         16, 32, 64, 128 or 256;  num_pages * kv_heads * page_size below 2^31
 * Formats, for a row x of head_dim values (H the head_dim-point Hadamard
 * transform, adds in strides 1, 2, 4, ... in fp32):
 *   EXL3_KV_F16, EXL3_KV_BF16  x itself
 *   EXL3_KV_INT8   y = H x / 8;  scale = max|y| / 127 in fp32 (times the rounded reciprocal), rounded
 *                  up to bf16, at least 2^-100, 1 for a row of zeros;  code = rint(y * (1 / scale)),
 *                  stored as code + 128 in a byte
 *   EXL3_KV_INT4   the same with 7 in place of 127, code + 8 in a nibble, even values low
 * A row with a NaN or an infinity gets zero codes and a NaN scale and reads back as NaN.  The values read back are
 * H(codes) * scale * 8 / head_dim.  Attention works on the rotated rows: it
 * rotates q and its output instead.  Over a quantised cache its operands are fp16
 * in that basis, in units of powers of two taken from the rows themselves, so rows of any size
 * do.  Two limits: where max_q * (q_heads / kv_heads) is above 16, a row whose scale is 2^24 times below the largest
 * of the 16 keys (counted from a multiple of 16) that it lies among loses bits; and value scales that one query sees
 * may differ by a factor of 2^100 (a row of zeros, whatever its stored scale, may lie beside scales up to 2^40).
 */
typedef enum { EXL3_KV_F16 = 0, EXL3_KV_BF16 = 1, EXL3_KV_INT8 = 2, EXL3_KV_INT4 = 3 } exl3_kv_format_t;
typedef struct {
  void* k;
  void* v;
  uint16_t* k_scale;
  uint16_t* v_scale;
  int64_t num_pages;
  int32_t page_size, kv_heads, head_dim;
  exl3_kv_format_t format;
} exl3_kv_cache_t;

/*
 * exl3_kv_write -- write the key and value rows of `tokens` tokens into their
 * slots; with `rope`, keys are rotated on the way (rounded to the type, then
 * quantised), and so are the q_heads heads of q, into q_out: one launch for a
 * decode step.  rope NULL: nothing is rotated, and q, q_out are not used
 * (q_heads 0).  A 16-bit cache's format must be the rows' type.
 *   slots  device, int64 [tokens]: a slot outside the cache (a padding token's -1) writes nothing;
 *          no two tokens of a call share a slot
 *   q_out  device, may be q's own data (in place); may not overlap k or v
 */
exl3_status_t exl3_kv_write(const exl3_kv_cache_t* cache, const exl3_heads_t* k, const exl3_heads_t* v,
                            exl3_dtype_t dtype, int64_t tokens, const int64_t* slots, const exl3_rope_t* rope,
                            const exl3_heads_t* q, int32_t q_heads, void* q_out, int64_t q_out_token_stride,
                            int64_t q_out_head_stride, void* stream);

/*
 * exl3_norm_kv_write -- the same with the norms of exl3_norm_rope on the heads of
 * q and k (either may be NULL: none) and the axes of its positions.  A key's row
 * is normed, rotated, rounded to the type, then quantised.  q is taken if there
 * is something to do with it: q_heads > 0 needs rope or q_norm.
 */
exl3_status_t exl3_norm_kv_write(const exl3_kv_cache_t* cache, const exl3_heads_t* k, const exl3_heads_t* v,
                                 exl3_dtype_t dtype, int64_t tokens, const int64_t* slots,
                                 const exl3_head_norm_t* q_norm, const exl3_head_norm_t* k_norm,
                                 const exl3_rope_t* rope, const exl3_rope_axes_t* axes, const exl3_heads_t* q,
                                 int32_t q_heads, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                                 void* stream);

/*
 * exl3_kv_read -- the rows of `tokens` slots, as `dtype` (each one rounding of
 * the value read back).  A slot outside the cache reads as zeros.
 *   k, v  device, [tokens][kv_heads][head_dim] (outputs)
 */
exl3_status_t exl3_kv_read(const exl3_kv_cache_t* cache, const int64_t* slots, int64_t tokens,
                           exl3_dtype_t dtype, void* k, void* v, void* stream);

/*
 * Page tables of a batch of requests, kept on the GPU, with the free pages as a
 * stack.  Request b's row of block_table holds its first held[b] pages (which may be more than its kv_lens[b]
 * cached tokens fill: a length may be set back, when drafted tokens are refused, without giving pages back).
 *   block_table  device, int32 [batch][table_width];  table_width * page_size at most 2^30
 *   kv_lens, held  device, int32 [batch]
 *   free_pages   device, int32 [capacity]: the free pages are its first free_count[0] entries;  capacity below 2^30
 *   page_size    as for the cache
 * What lies outside its range (a length above table_width * page_size, a count above capacity) is taken as the
 * nearest that does not.
 */
typedef struct {
  int32_t* block_table;
  const int32_t* kv_lens;
  const int32_t* held;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t batch, table_width, page_size, capacity;
} exl3_kv_tables_t;

/*
 * exl3_kv_plan -- a step's packing, positions and slots from the number of new
 * tokens of each request, and pages for them: one launch, no host copy.
 *   n_b = max(0, new_lens[b]);  cu_q[b] = min(total, sum of n before b), cu_q[batch] likewise of all
 *   need_b = max(0, ceil((kv_lens[b] + n_b) / page_size) - held[b]), 0 where n_b = 0
 *   a request can be served if its rows lie below total and its pages fit into table_width.  One that can and
 *   needs no page is granted; one that needs some is granted if its need and those of all requests before it that
 *   can be served are at most free_count (so none overtakes one that waits for pages)
 * Granted: its new pages come from the top of the stack, in order, into its row of the table; kv_lens_out =
 * kv_lens + n, held_out = held + need.  Row cu_q[b] + i has position kv_lens[b] + i and the slot of that position.
 * Not granted: length, pages and table stay; its rows have positions as above and the slot -1, which exl3_kv_write
 * skips.  Rows from cu_q[batch] to total (padding of a captured step): position 0, slot -1.
 * Attention over the new state takes the rows of a request that was not granted for the last tokens of its old
 * length: what it gives for them means nothing.
 *   new_lens  device, int32 [batch]
 *   kv_lens_out, held_out, free_count_out  device (outputs): the new state; may be the tables' own (updated in place)
 *   cu_q      device, int32 [batch + 1];  positions  int32 [total];  slots  int64 [total];  granted  uint8 [batch], 0 or 1
 * Entries of block_table from held on, and free_pages above the stack, are never read.
 */
exl3_status_t exl3_kv_plan(const exl3_kv_tables_t* tables, const int32_t* new_lens, int64_t total,
                           int32_t* kv_lens_out, int32_t* held_out, int32_t* free_count_out, int32_t* cu_q,
                           int32_t* positions, int64_t* slots, uint8_t* granted, void* stream);

/*
 * exl3_kv_release -- requests end: their pages go onto the stack (in order of the
 * requests, a row's pages in order; those past capacity are dropped), their
 * lengths and held pages become 0; others keep theirs.  The table's entries stay.
 *   ended   device, uint8 [batch]: not 0 where the request ends
 *   shared  device, int32 [batch], may be NULL: leading pages of an ended request that are not its own and stay out
 *           of the stack
 *   other arguments as for exl3_kv_plan
 */
exl3_status_t exl3_kv_release(const exl3_kv_tables_t* tables, const uint8_t* ended, const int32_t* shared,
                              int32_t* kv_lens_out, int32_t* held_out, int32_t* free_count_out, void* stream);

/*
 * exl3_attention_prompt -- causal attention over whole prompts, packed one
 * after the other:
 *     out[i] = sum_j p_ij v[j] / sum_j p_ij,  p_ij = exp(scale * q[i] . k[j])
 * over the keys j <= i of i's own sequence and, with window > 0, j > i - window.
 * Scores, softmax statistics and sums are fp32; the weights round to the type
 * before they meet v.
 *   q, k, v    [total] tokens of `dtype`;  scale  positive and finite
 *   v          a value that is not finite may also reach those queries of its sequence that do not see it (a weight
 *              of zero still multiplies it), never another sequence
 *   cu_seqlens device, int32 [batch + 1]: sequence b is tokens [cu[b], cu[b + 1]); tokens of no
 *              sequence keep their output
 *   out        device, [total] tokens of q_heads heads; may be q itself (same strides), else it overlaps
 *              no input
 */
exl3_status_t exl3_attention_prompt(const exl3_heads_t* q, const exl3_heads_t* k, const exl3_heads_t* v,
                                    exl3_dtype_t dtype, int64_t total, int32_t q_heads, int32_t kv_heads,
                                    int32_t head_dim, const int32_t* cu_seqlens, int32_t batch, int32_t window,
                                    float scale, void* out, int64_t out_token_stride, int64_t out_head_stride,
                                    void* stream);

/*
 * exl3_attention_paged -- the same over the cache, for the last tokens of each
 * sequence (one, a few drafted ones, or a chunk of a prompt), whose keys and
 * values are already written.  Query i of sequence b stands at position
 * kv_lens[b] - (cu_q[b + 1] - cu_q[b]) + i and sees the keys up to its own; a
 * query that sees none (a negative position, an empty sequence) gives zeros.
 *   q           [total_q] tokens of `dtype` (a 16-bit cache's format must be the same)
 *   block_table device, int32 [batch][table_width]: pages of a sequence in order.  Entries past the
 *               length are not followed; with a window neither are those of pages wholly before it.  An entry
 *               outside the cache is not followed either (its keys count as zeros)
 *   cu_q        device, int32 [batch + 1]: query tokens of sequence b, as cu_seqlens above
 *   kv_lens     device, int32 [batch]: cached tokens, the new ones among them; at most table_width * page_size
 *   out         as for exl3_attention_prompt
 *   batch       times kv_heads below 2^31
 *   max_q       HOST: no sequence has more query tokens (the outputs of one that has are undefined)
 *   max_kv      HOST: about the longest length; it only steers how the work is split
 *   workspace   device, 16-byte aligned, at least exl3_attention_paged_workspace_bytes of the same sizes
 *               (0 bytes: may be NULL), any contents.  Calls that share it must be ordered on one stream.
 * Values (and value scales) of keys that one query of a call may not see but another of the same sequence
 * does must be finite: a weight of zero still multiplies them.  Rows past a length, and rows before the first that a
 * query of the call sees, may hold anything.
 * If a kernel gives up on a bounded wait (exl3_device_status reports it), out is undefined.
 */
size_t exl3_attention_paged_workspace_bytes(int64_t total_q, int32_t batch, int32_t q_heads, int32_t kv_heads,
                                            int32_t head_dim, int32_t max_q, int32_t max_kv, int32_t window);
exl3_status_t exl3_attention_paged(const exl3_heads_t* q, exl3_dtype_t dtype, int64_t total_q, int32_t q_heads,
                                   const exl3_kv_cache_t* cache, const int32_t* block_table, int32_t table_width,
                                   const int32_t* cu_q, const int32_t* kv_lens, int32_t batch, int32_t max_q,
                                   int32_t max_kv, int32_t window, float scale, void* out,
                                   int64_t out_token_stride, int64_t out_head_stride, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * exl3_attention_shared -- exl3_attention_paged (without a window) for sequences
 * that begin with the same cached tokens (one system prompt, one document, several
 * answers to one question): keys and values of what a group of sequences shares are read once for all of it.
 * Group g is the sequences cu_groups[g] .. cu_groups[g + 1] - 1, whose first prefix_lens[g] keys and values are the
 * same.  They are read through the block table of the group's first sequence that has queries; usually the
 * sequences' tables name the same pages, but copies (of a last page that is filled up differently) will do.
 * Sequences of no group (before cu_groups[0], from cu_groups[groups] on) are as in exl3_attention_paged.
 * Where the sizes say that sharing does not pay (few sequences, short prefixes), the call is exl3_attention_paged.
 * The result is exl3_attention_paged's but for the order of its sums and, where prefixes of a quantised cache are
 * shared, the roundings that it has in long chunks: the rotated q is one fp16 term, and every key and value of the
 * prefix (code times scale) an fp16 number.  (For few rows the paged call takes codes as they are, scales in fp32 and
 * q of fp16 rows in two terms; such fp16 rows are not shared unless EXL3_SHARE_ALWAYS asks for it.)
 * What is shared in fact is whole tiles of 128 keys that every query of the group sees, from 256 keys on, of groups
 * in which at least two sequences have queries: prefix_lens may be larger than a sequence's length or reach past a
 * query's position.  So the sequence that sees least says how much its group shares: n rows that exl3_kv_plan did
 * not grant, behind a prefix that is all that is cached, take n - 1 keys off it, or all.
 *   cu_groups    device, int32 [groups + 1], not falling;  prefix_lens  device, int32 [groups]
 *   max_prefix   HOST: about the longest prefix; it steers whether prefixes are shared.
 *                EXL3_SHARE_ALWAYS: they are, whatever the sizes say; 0: they are not.  The sizes are weighed as if
 *                every sequence were of a group: where the groups hold fewer, ask exl3_attention_shared_pays
 *   workspace    as for exl3_attention_paged, at least exl3_attention_shared_workspace_bytes of the same sizes
 *   other arguments and limits as for exl3_attention_paged
 */
#define EXL3_SHARE_ALWAYS INT32_MAX
size_t exl3_attention_shared_workspace_bytes(int64_t total_q, int32_t batch, int32_t groups, int32_t q_heads,
                                             int32_t kv_heads, int32_t head_dim, exl3_dtype_t dtype,
                                             exl3_kv_format_t format, int32_t max_q, int32_t max_kv, int32_t max_prefix);
/* 1 where the sizes say that sharing pays for groups that hold `sharers` of the batch's sequences, else 0 (also for sizes
 * that the call refuses).  Where it is 0, pass max_prefix 0. */
int32_t exl3_attention_shared_pays(int64_t total_q, int32_t batch, int32_t sharers, int32_t groups, int32_t q_heads,
                                   int32_t kv_heads, int32_t head_dim, exl3_dtype_t dtype, exl3_kv_format_t format,
                                   int32_t max_q, int32_t max_prefix);
exl3_status_t exl3_attention_shared(const exl3_heads_t* q, exl3_dtype_t dtype, int64_t total_q, int32_t q_heads,
                                    const exl3_kv_cache_t* cache, const int32_t* block_table, int32_t table_width,
                                    const int32_t* cu_q, const int32_t* kv_lens, int32_t batch, const int32_t* cu_groups,
                                    const int32_t* prefix_lens, int32_t groups, int32_t max_q, int32_t max_kv,
                                    int32_t max_prefix, float scale, void* out, int64_t out_token_stride,
                                    int64_t out_head_stride, void* workspace, size_t workspace_bytes, void* stream);

/*
 * exl3_gemm_splitk_noalloc -- the split-k GEMM for callers that cannot allocate.
 *
 * The pages have no counterpart to this call; it exists for callers that have
 * no way to obtain a device workspace (a plugin inside a host program that owns
 * the allocator, or code that must not call cudaMalloc because it would
 * synchronise the device or break a fixed memory budget).  It computes exactly
 * what exl3_gemm_splitk computes, with the same arguments minus the workspace:
 * the fp32 partials go to a scratch array built into the library, of
 * EXL3_NOALLOC_SCRATCH_BYTES per GPU, held on every GPU that loads the library
 * until the process exits.  It calls no allocator.
 *
 *  - Size limit: exl3_splitk_workspace_bytes(m, k, n) must not exceed
 *    EXL3_NOALLOC_SCRATCH_BYTES; a larger request returns EXL3_EWORKSPACE and
 *    launches nothing (use exl3_gemm_splitk with your own workspace instead).
 *  - Each call looks up the scratch array's address in the current device's
 *    context (a lookup that allocates nothing), so no address outlives a
 *    context: after cudaDeviceReset the next call uses the new context's array.
 *    Loading the module on a device happens at its first call; make that call
 *    before any stream capture on that device.
 *  - Every call shares the one array.  Calls whose work may overlap on the GPU
 *    (different streams, or different threads without ordering) race on it and
 *    give wrong results; order them on one stream.  Each call overwrites every
 *    partial it reads, so what an earlier call left behind does no harm.
 *  - As for exl3_gemm_splitk, y is undefined for a call during which
 *    exl3_device_status records a wait that gave up.
 */
#define EXL3_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
exl3_status_t exl3_gemm_splitk_noalloc(const uint16_t* xh, int64_t m, int64_t k, const int16_t* trellis,
                                       int32_t bits, exl3_codebook_t cb, const uint16_t* svh,
                                       const int32_t* shard_cols, int32_t num_shards, void* y,
                                       exl3_dtype_t y_dtype, int64_t n, void* stream);

/*
 * Test-only entry points (they run the same device decode as exl3_gemm).
 *
 * exl3_test_codebook: out[s] = fp16 bits of codebook cb at state s, s = 0..65535
 *   (TensorFold PR #740, "Tests": all 65,536 states of each codebook).  The
 *   library decodes with two instruction sequences (one per kernel family);
 *   a state where they disagree reads 0xFFFF, a NaN no state decodes to.
 *   out: device, uint16 [65536].
 * exl3_test_unpack: wq[k][n] = decoded weights of the whole trellis as fp16 bits
 *   (TensorFold PR #740, "Tests": random tiles at every width and codebook).
 *   trellis: device int16 [k/16][n/16][16*bits]; wq: device uint16 [k][n].
 *   k and n need only be multiples of 16 here.
 */
exl3_status_t exl3_test_codebook(exl3_codebook_t cb, uint16_t* out, void* stream);
exl3_status_t exl3_test_unpack(const int16_t* trellis, int32_t bits, exl3_codebook_t cb,
                               int64_t k, int64_t n, uint16_t* wq, void* stream);

/*
 * exl3_test_gemm_shape: exl3_gemm (acc == NULL) or exl3_gemm_splitk (acc !=
 * NULL, same workspace rules) with the kernel's tile shape fixed by the caller
 * instead of chosen from the call's sizes.  Every tile shape computes each
 * output element with the same k16 steps in the same order, so the result must
 * be byte-equal to the one the library picks; tests use this to check each
 * shape.  No counterpart in the pages: the tiling is this library's own.
 *   tile_shape: 0 = 32-column strips (m <= 32, k/128 even, no split-k),
 *     1 = 64-column strips (m <= 32), 2 = 128 columns (m <= 32),
 *     3 = 128 columns x 128 rows, 4 = 128 columns x 256 rows,
 *     5 = 256 columns x 256 rows (n and shard edges multiples of 256),
 *     6 = pair of 128-column x 256-row CTAs sharing decoded weights,
 *     7 = pair of 256-column x 256-row CTAs (edges multiples of 256),
 *     8 = 128 columns, four k atoms per stage (m <= 32, k/128 even, no split-k),
 *     9 = 96-column strips in clusters of four CTAs over three Hadamard blocks
 *         (m <= 32, k/128 even, no split-k, n and shard edges multiples of 384),
 *     10 = 96 columns x 128 rows, 11 = 96 columns x 256 rows (clusters of four
 *         as in 9; n and shard edges multiples of 384),
 *     12 = 32-column strips with eight k atoms per stage (m <= 32, k a
 *         multiple of 512, no split-k), 13 = 64-column strips with four
 *         (m <= 32, k/128 even, no split-k), 14 = 96-column strips holding
 *         64 rows with four (m <= 64, k/128 even, no split-k, n and shard
 *         edges multiples of 384), 15 = 64-column strips holding 64 rows with
 *         four (m <= 64, k/128 even, no split-k), 16 = 64-column strips of
 *         128 rows with four (k/128 even, no split-k), 17 = 32-column strips
 *         of 128 rows with four (k/128 even, no split-k).
 *     The decoded weights as the tensor core's 128-row operand and the batch
 *     rows as the narrow one (18, 19, 21, 23 keep the decoded weights in
 *     tensor memory, 20 and 22 in shared memory):
 *     18 = 128 columns, four k atoms per stage (m <= 32, k/128 even; under
 *         split-k only when its parts are whole 256-row units of k), 19 =
 *         128 columns, two k atoms (m <= 32), 20 = 96-column
 *         strips in clusters of four, four k atoms (m <= 32, k/128 even, no
 *         split-k, n and shard edges multiples of 384), 21 and 22 = 18 and 20
 *         holding 16 rows (m <= 16), 23 = 19 holding 16 rows (m <= 16),
 *         24 = 18 holding 64 rows (m <= 64), 25 = 19 holding 64 rows
 *         (m <= 64), 26 = 19 holding 128 rows (m <= 128), 27 = 20 holding
 *         64 rows (m <= 64), 28 = 18 holding 128 rows (m <= 128; two k
 *         atoms per stage at 7-8 bits).
 * Returns EXL3_EUNSUPPORTED, launching nothing, when the shape cannot run the
 * call (the conditions in parentheses).
 */
#define EXL3_TEST_TILE_SHAPES 29
exl3_status_t exl3_test_gemm_shape(int32_t tile_shape, const uint16_t* xh, int64_t m, int64_t k,
                                   const int16_t* trellis, int32_t bits, exl3_codebook_t cb,
                                   const uint16_t* svh, const int32_t* shard_cols, int32_t num_shards,
                                   void* y, exl3_dtype_t y_dtype, int64_t n, float* acc, size_t acc_bytes,
                                   void* stream);

/*
 * exl3_test_tile_plan: the cost model's plan for an exl3_gemm call (split = 0)
 * or exl3_gemm_splitk call (split = 1) of the given sizes, computed on the host
 * with no launch (the SM count of the current device, 152 when there is none).
 * out[0] = tile shape (numbered as in exl3_test_gemm_shape); for a pair shape
 * whose partial last wave runs as a second launch of smaller tiles (or of
 * 128-column pairs), out[1] =
 * that launch's shape, out[2] = pair tiles of the first launch, out[3] and
 * out[4] = first row and first column of the second launch; otherwise
 * out[1] = -1 and out[2..4] = 0.  EXL3_EINVAL for invalid sizes or shard map.
 * No counterpart in the pages: the tiling is this library's own.
 */
exl3_status_t exl3_test_tile_plan(int64_t m, int64_t k, int64_t n, const int32_t* shard_cols, int32_t num_shards,
                                  int32_t split, int64_t* out);

/*
 * Tile-shape autotune (off by default).  The best tile for a batch size
 * depends on the layer's shape too, so the shape is timed once per distinct
 * shape and cached, never while a CUDA graph is being captured, and the cost
 * model stays the fallback for captured work (cuda-exl3 README, "Where the
 * time goes").  Here the split-k parts are fixed by (k, n) so that rows stay
 * byte-equal across batch sizes; only the tile shape is tuned.
 * When enabled, the first uncaptured exl3_gemm / exl3_gemm_splitk call of each
 * key (device, width, codebook, k, n, shard edges, split parts, batch bucket:
 * m <= 32, else the next power of two of m) times every tile shape that can
 * run it on the caller's stream, synchronising the host, and caches the
 * fastest (the cost model's shape unless another is more than 2% faster).
 * The timing launches write the call's own y (or acc) several times; the
 * result is the final launch's, and every shape computes the same bytes, so
 * tuning never changes a result.  A call under capture uses the cached shape
 * of its key if there is one (tune in an eager warm-up to reach captured
 * work), else the cost model's, and never tunes.
 *   exl3_set_autotune(1 | 0): EXL3_EINVAL for any other value.
 *   exl3_clear_autotune(): forget every cached key.
 *   exl3_autotune_entries(): the number of cached keys.
 */
exl3_status_t exl3_set_autotune(int32_t enable);
exl3_status_t exl3_clear_autotune(void);
int64_t exl3_autotune_entries(void);

/*
 * exl3_device_status -- read and clear the library's device-side error flags.
 * Every wait inside the kernels is bounded; a kernel that gives up sets bit 0
 * (EXL3_DEVERR_WAIT_TIMEOUT) and skips its stores instead of hanging.  This call
 * synchronises the current device (it is meant for tests and diagnostics).
 *   flags: host pointer, receives the OR of all flags set since the last call.
 */
#define EXL3_DEVERR_WAIT_TIMEOUT 1u
exl3_status_t exl3_device_status(uint32_t* flags);

/*
 * exl3_test_wait_timeout -- test-only: the failure path of the bounded waits.
 * One CTA waits, with the same bounded mbarrier wait every kernel of the
 * library uses, on a barrier that nothing arrives on.  The wait gives up after
 * 2 s, the kernel sets EXL3_DEVERR_WAIT_TIMEOUT (read by exl3_device_status)
 * and writes *out = 0 (1 would mean the wait had returned).  It faults
 * nothing and leaves the context usable.  No counterpart in the pages.
 *   out: device uint32, 4-byte aligned; EXL3_EINVAL when null or misaligned.
 */
exl3_status_t exl3_test_wait_timeout(uint32_t* out, void* stream);

/* Static text for a status code. */
const char* exl3_status_string(exl3_status_t status);
/* Text of the last CUDA error seen by this thread's calls ("" if none). */
const char* exl3_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* EXL3_H */
