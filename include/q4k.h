/*
 * q4k.h -- C ABI of the GB300 (sm_103a) Q4_K decode library.
 *
 * The library computes the memory-bound decode products of a GGUF Q4_K_M
 * engine directly on 4-bit block-quantized weights:
 *   - q4k_gemv         y = W x for one token or a small batch of tokens
 *                      ("custom quantized GEMV for decode (Q8_0, Q4_K, Q6_K)"
 *                      with "on-the-fly weight dequantization", dotLLM README,
 *                      News 2026-03 "CUDA GPU backend"; the batch form is the
 *                      VerifyBatch pass of the Glacier.Inference article,
 *                      section 4 "Beating Hardware Bandwidth Ceilings with
 *                      Speculative Decoding": one weight read for K+1 tokens)
 *   - q4k_gemv_argmax  the LM-head product fused with a greedy argmax that
 *                      writes one int32 token id per batch row (Glacier.Inference
 *                      article, section 2 "Eliminating PCIe Starvation: In-VRAM
 *                      Warp-Shuffle Argmax")
 *   - q4k_gemm_prefill the prefill product with bf16 activations ("cuBLAS HGEMM
 *                      for prefill", dotLLM README, News 2026-03), here on the
 *                      tcgen05 tensor cores after a dequantize-to-fp16 step
 *                      (q4k_gemm_prefill_exact: the same with exact integer
 *                      weight tiles).
 *   - q6k_gemv         y = W x for a Q6_K matrix, the other block format of
 *                      Q4_K_M files ("custom quantized GEMV for decode (Q8_0,
 *                      Q4_K, Q6_K)", same page and item); q6k_repack_planar
 *                      and q6k_gemv_planar: the same product on a copy of
 *                      the matrix split into aligned planes once, at load
 *                      time (the dotLLM README repacks its weights at model
 *                      load time too: News 2026-03, the R4 row interleave).
 *
 * ---------------------------------------------------------------------------
 * Q4_K super-block (144 bytes, 256 weights, 4.5 bits per weight)
 * ---------------------------------------------------------------------------
 * The pages name the format (Q4_K, Q4_K_M) but print no byte layout; this
 * library fixes the GGUF Q4_K packing:
 *   bytes   0..1   d     IEEE binary16, little-endian (super-block scale)
 *   bytes   2..3   dmin  IEEE binary16, little-endian (super-block min scale)
 *   bytes   4..15  s[12] eight 6-bit scales sc_j and eight 6-bit mins m_j:
 *                    j < 4 : sc_j = s[j] & 63,  m_j = s[j+4] & 63
 *                    j >= 4: sc_j = (s[j+4] & 15) | ((s[j-4] >> 6) << 4)
 *                            m_j  = (s[j+4] >> 4) | ((s[j]   >> 6) << 4)
 *   bytes  16..143 qs[128] 4-bit quants; for p = 0..3 and i = 0..31:
 *                    q[64p + i]      = qs[32p + i] & 15   (sub-block 2p)
 *                    q[64p + 32 + i] = qs[32p + i] >> 4   (sub-block 2p+1)
 *   weight 32j + i of the block:   w = d * sc_j * q[32j+i] - dmin * m_j
 *
 * A matrix W of N rows and K columns (K a positive multiple of 256) is stored
 * row-major as N rows of K/256 consecutive super-blocks: row n starts at byte
 * n * (K/256) * 144.  Every row therefore starts on a 16-byte boundary when W
 * does.
 *
 * ---------------------------------------------------------------------------
 * Conventions for every entry point
 * ---------------------------------------------------------------------------
 *   - All data pointers are DEVICE pointers owned by the caller; the library
 *     never frees or retains them.  Calls are asynchronous on `stream` (a
 *     cudaStream_t passed as void*; NULL is the legacy default stream) and
 *     never synchronize the host.
 *   - Outputs are overwritten, never accumulated.  Inputs and outputs must not
 *     overlap.
 *   - Argument errors are detected on the host before anything is launched and
 *     returned as a status; Q4K_ERR_CUDA reports a launch failure (the CUDA
 *     error is left for cudaGetLastError to clear).
 *   - x and X are read only inside the kernels; they may be produced by the
 *     kernel that ran just before on the same stream.
 */
#ifndef Q4K_H
#define Q4K_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define Q4K_BLOCK_WEIGHTS 256
#define Q4K_BLOCK_BYTES 144
#define Q4K_MAX_BATCH 16
#define Q4K_ABI_VERSION 1

typedef enum {
    Q4K_OK = 0,
    Q4K_ERR_INVALID_ARG = 1,        /* null pointer, bad size or batch */
    Q4K_ERR_MISALIGNED = 2,         /* a pointer is not 16-byte aligned */
    Q4K_ERR_UNSUPPORTED_DEVICE = 3, /* current device is not compute capability 10.3 */
    Q4K_ERR_CUDA = 4                /* a CUDA call or a launch failed */
} q4k_status;

/* Human-readable text of a status (static storage, never NULL). */
const char *q4k_status_string(q4k_status s);

/* Q4K_ABI_VERSION of the loaded library. */
int q4k_abi_version(void);

/*
 * y[b][n] = sum_k w[n][k] * x[b][k]   for b < batch, n < N.
 *   W     uint8  [N][K/256*144]  Q4_K rows (layout above), 16-byte aligned
 *   x     fp32   [batch][K]      row-major, 16-byte aligned
 *   y     fp32   [batch][N]      row-major
 *   N >= 0 (N == 0 is a no-op and W, y may then be NULL), K a positive multiple
 *   of 256, K/256 < 2^24, 1 <= batch <= 16.
 * Accumulation is fp32.  Each weight super-block is read from memory once for
 * all batch rows.  x may hold any finite fp32 values.  Inside, each
 * super-block of x is carried in one of two forms:
 *   - batch 1: two int8 parts, x ~= (a/32258)(254 xh + xl) with a = max|x| of
 *     the super-block (error <= a (1/64516 + 2^-16)); the weight nibbles are
 *     multiplied with them by integer dot products (dp4a), exact in int32,
 *     and the scales applied per super-block in fp32;
 *   - batch >= 2 (and batch 1 with Q4K_FLAG_TENSOR_CORE): two fp16 parts after
 *     a power-of-two scale (error <= 2^-22 |x|), multiplied with the weights as
 *     exact fp16 integers on the tensor cores (mma.sync), fp32 accumulation.
 * Errors: INVALID_ARG (null pointer, N < 0, K <= 0 or K % 256 != 0, batch out
 * of range), MISALIGNED (W or x), UNSUPPORTED_DEVICE, CUDA.
 */
q4k_status q4k_gemv(const void *W, const float *x, float *y, int64_t N, int64_t K, int batch,
                    void *stream);

/*
 * idx[b] = the smallest n with y[b][n] == max_n' y[b][n'], where y = W x is the
 * product q4k_gemv computes (the very same fp32 values).  NaN never wins; a row
 * whose values are all NaN gives 0; -0.0 and +0.0 compare equal.  No logits
 * leave the device: the only output is batch int32 values.
 *   idx   int32 [batch]
 *   1 <= N <= 2^31 - 1; other arguments as for q4k_gemv.
 * Scratch: 144 bytes taken from the stream-ordered allocator (cudaMallocAsync,
 * cleared with cudaMemsetAsync, released with cudaFreeAsync, all on `stream`),
 * so concurrent calls on different streams are independent.
 */
q4k_status q4k_gemv_argmax(const void *W, const float *x, int32_t *idx, int64_t N, int64_t K,
                           int batch, void *stream);

/*
 * Same as q4k_gemv_argmax, and also writes the logits it reduced to
 * `logits` (fp32 [batch][N]); meant for tests that check the argmax bit for bit
 * against a scan of the very values the kernel compared.
 */
q4k_status q4k_gemv_argmax_debug(const void *W, const float *x, int32_t *idx, float *logits,
                                 int64_t N, int64_t K, int batch, void *stream);

/*
 * Allocation-free q4k_gemv_argmax.  (No counterpart on the pages: this is an
 * interface choice of this library.)  Same arguments, same result bit for bit.
 * Meant for callers that must not allocate device memory while they run --
 * code working from a fixed, pre-sized memory budget, real-time loops that
 * forbid allocator calls, or processes whose stream-ordered allocator is
 * unavailable or replaced.  Instead of cudaMallocAsync it uses a static device
 * array of 16 keys + a ticket (144 bytes) that every GPU loading the library
 * keeps until the process exits.
 *   - batch must be <= 16 (the array's capacity); larger batches return
 *     Q4K_ERR_INVALID_ARG.
 *   - The array's device address is looked up (cudaGetSymbolAddress) on the
 *     first call on a device and on every call made outside stream capture;
 *     a call made during capture reuses the last address looked up, so make a
 *     first call on each device before any stream capture (and again after a
 *     cudaDeviceReset, which may move the array).
 *   - Each call clears the array with cudaMemsetAsync on `stream` before its
 *     kernel.  All calls share the array: calls that overlap on the GPU
 *     (different streams, concurrently running graphs) race and may return
 *     wrong indices.  Serialize them.
 *   - Allocates nothing: no cudaMalloc, cudaMallocAsync or cudaFree.
 */
q4k_status q4k_gemv_argmax_noalloc(const void *W, const float *x, int32_t *idx, int64_t N, int64_t K,
                                   int batch, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Q6_K super-block (210 bytes, 256 weights, 6.5625 bits per weight), the other
 * block format of Q4_K_M files ("custom quantized GEMV for decode (Q8_0, Q4_K,
 * Q6_K)", dotLLM README, News 2026-03 "CUDA GPU backend").  The pages print no
 * bytes; this library fixes the GGUF Q6_K packing:
 *   bytes   0..127  ql[128] low 4 bits of the 6-bit codes
 *   bytes 128..191  qh[64]  high 2 bits of the codes
 *   bytes 192..207  sc[16]  int8 scale of each 16 weights
 *   bytes 208..209  d       IEEE binary16, little-endian
 *   weight k = 128h + 32c + l (h < 2, c < 4, l < 32):
 *     low  = ql[64h + 32(c & 1) + l], its low nibble for c < 2, high for c >= 2
 *     high = (qh[32h + l] >> 2c) & 3,   q = low + 16 high (0..63)
 *     w = d * sc[k / 16] * (q - 32)
 * Rows hold K/256 consecutive blocks (row n at byte n * (K/256) * 210); blocks
 * are therefore only 2-byte aligned.
 * ---------------------------------------------------------------------------
 * y[b][n] = sum_k w[n][k] * x[b][k] for a Q6_K matrix W, b < batch, n < N.
 *   W uint8 [N][K/256*210] (16-byte aligned), x fp32 [batch][K] (16-byte
 *   aligned), y fp32 [batch][N]; N >= 0 (0: no-op), K a positive multiple of
 *   256, 1 <= batch <= 16.  Each block is read once for all batch rows;
 *   deterministic.  For batch <= 4 and K <= 4096, whole 8-row tiles take an
 *   integer inner product: x enters per 256-block as two int8 parts
 *   (x ~ (a/32258)(254 xh + xl), a = the block's max |x|, error <=
 *   a (1/64516 + 2^-16) per element), the weight codes meet them in exact
 *   int32 dot products and the scales in fp32; the other rows and shapes
 *   multiply in fp32.  Both stay far inside the stated tolerance.
 * Errors: INVALID_ARG, MISALIGNED (W or x), UNSUPPORTED_DEVICE, CUDA.
 */
q4k_status q6k_gemv(const void *W, const float *x, float *y, int64_t N, int64_t K, int batch, void *stream);

/*
 * Planar Q6_K: the bytes of a Q6_K matrix regrouped so that every block's
 * codes and scales start on a 16-byte boundary (GGUF blocks are only 2-byte
 * aligned), for the GEMV below.  For N rows and nb = K/256 blocks per row,
 * with DP = 2*nb rounded up to a multiple of 16, the planar buffer holds
 *   QS  [N][nb][208]  bytes 0..207 of each block (ql, qh, sc), unchanged
 *   D   [N][DP]       d of block j at bytes 2j, 2j+1 of the row; the rest 0
 * QS at byte 0 and D at byte N*nb*208, q6k_planar_bytes(N, K) =
 * N * (nb*208 + DP) bytes in all (2940 + 4 bytes per row for K = 3584).  The
 * weights it encodes are exactly those of the GGUF matrix.  Returns -1 for
 * N < 0 or K not a positive multiple of 256.
 */
int64_t q6k_planar_bytes(int64_t N, int64_t K);

/*
 * Wp = the planar form of the Q6_K matrix W (above).  W uint8 [N][K/256*210]
 * (16-byte aligned); Wp device memory of q6k_planar_bytes(N, K) bytes
 * (16-byte aligned), not overlapping W; asynchronous on stream.  N >= 0 (0:
 * no-op), K a positive multiple of 256.  Errors: INVALID_ARG, MISALIGNED,
 * UNSUPPORTED_DEVICE, CUDA.
 */
q4k_status q6k_repack_planar(const void *W, void *Wp, int64_t N, int64_t K, void *stream);

/*
 * y = W x as q6k_gemv computes it, from the planar form Wp of W: the same
 * arguments, with Wp (q6k_planar_bytes(N, K) bytes, 16-byte aligned) in place
 * of W.  Every block is read once for all batch rows.  The planes stream into
 * shared memory as 2-D TMA boxes of 128 rows (one block per stage), so each
 * thread reads its codes, scales and d with 16-byte loads; x enters per
 * 256-block as the two int8 parts of q6k_gemv's integer path and the codes
 * meet them in exact int32 dot products (batch rows 1..8 per launch; larger
 * batches take one launch per eight rows).  Deterministic; K splits over the
 * CTAs of a cluster add their partial rows in rank order.
 * Errors: INVALID_ARG, MISALIGNED (Wp or x), UNSUPPORTED_DEVICE, CUDA.
 */
q4k_status q6k_gemv_planar(const void *Wp, const float *x, float *y, int64_t N, int64_t K, int batch,
                           void *stream);

/*
 * Y[t][n] = sum_k w[n][k] * X[t][k]   for t < T, n < N (prefill).
 *   W  Q4_K rows as above (16-byte aligned)
 *   X  bf16 [T][K] row-major (16-byte aligned)
 *   Y  fp32 [T][N] row-major
 * Up to 32 tokens this is q4k_gemm_prefill_exact (below: no weight is
 * rounded).  Above that each weight is dequantized in fp32 (one fma),
 * multiplied by a power of two chosen per row from the row's largest possible
 * |w|, and rounded to fp16 (nearest even) in shared memory; each token's
 * activations are converted to fp16
 * under a power of two chosen per token from its largest |x| (exact for every
 * value of at least 2^-31 times that largest).  The tcgen05 tensor cores
 * multiply them with fp32 accumulation in tensor memory and the epilogue
 * removes both scales.  Result: |Y - exact| <= ~2^-11 sum_k |w||x| for any
 * finite inputs, no overflow from large d, dmin or x.
 * Scratch: the converted X (2*T*K bytes), T scale exponents and, up to 32
 * tokens, T*K/2 bytes of sub-block sums come from cudaMallocAsync on `stream`
 * and are freed on it after the product.
 * Any T >= 0 is accepted (T == 0 or N == 0 is a no-op, and the pointers may
 * then be NULL); tokens go in tiles of 32 (T <= 32), 64 (T <= 64), 128, 256
 * or 512.
 * Errors: INVALID_ARG, MISALIGNED (W or X), UNSUPPORTED_DEVICE, CUDA
 * (including a failed scratch allocation).
 */
q4k_status q4k_gemm_prefill(const void *W, const void *X_bf16, float *Y, int64_t N, int64_t K,
                            int64_t T, void *stream);

/*
 * The same product with no weight rounding at all (arguments, layouts, errors
 * and scratch as q4k_gemm_prefill, plus T*K/2 bytes of scratch for the
 * sub-block sums of X).  The weight tiles hold q * sc_j, an integer of at most
 * 945 that fp16 represents exactly; the tensor cores accumulate
 * D = sum (q sc) x per super-block in tensor memory, one more MMA forms
 * M = sum_j m_j S_j from the sub-block sums S_j of the fp16 X (split into fp16
 * hi + lo), and y += d D - dmin M in fp32.  The only roundings are the fp32
 * accumulations and the hi + lo split of S_j.  Tiles of 32 (T <= 32) or 64
 * tokens; any T >= 0.  q4k_gemm_prefill takes this path up to 32 tokens;
 * from 33 tokens on the fp16 path is faster (14336 x 4096 at 64 tokens: 35.2
 * against 44.2 us), so this entry point is for callers that want the weights
 * exact there too.
 */
q4k_status q4k_gemm_prefill_exact(const void *W, const void *X_bf16, float *Y, int64_t N, int64_t K,
                                  int64_t T, void *stream);

/*
 * Extended launch control (tests and benchmarks).  Zero-initialised options
 * reproduce the plain entry points exactly.
 *   split_k  0 = automatic (up to 16 CTAs per tile for batch <= 8, when all
 *            clusters fit on the GPU at once); 1 <= s <= 8 forces the K range
 *            of every row tile to be split over s cooperating CTAs of a
 *            thread-block cluster (clamped to K/256).
 *   flags    Q4K_FLAG_PDL: launch with programmatic dependent launch, so the
 *            kernel may start streaming W while the previous kernel on the
 *            stream is still running.  W must then not be written by that
 *            previous kernel (weights are constant during decode); x is still
 *            read only after the previous kernel has completed.
 *            Q4K_FLAG_TENSOR_CORE: batch 1 uses the tensor-core inner product
 *            of the larger batches instead of the integer one.
 *            Q4K_FLAG_Q8K_X: batch 1 with x quantized Q8_K style (dotLLM README,
 *            News 2026-03 "Mixed quantization + Q8_K": 256-element blocks, a
 *            float32 scale, int8 codes, precomputed block sums): per block
 *            a = max|x|, d = a/127, q = rint(x * (127/a)) in fp32 (round half
 *            to even); the result is the product of W with d*q (exact integer
 *            dot products, fp32 per block), so it differs from W x by at most
 *            sum_k |w_k| d/2 per row -- its own tolerance, not the one stated
 *            for q4k_gemv.  Returns Q4K_ERR_INVALID_ARG with batch > 1 or
 *            together with Q4K_FLAG_TENSOR_CORE.
 *            Q4K_FLAG_TEST_STALL (failure-path tests only): the first weight
 *            copy of every CTA is awaited for 16 bytes more than it brings, so
 *            that every wait on it runs out.  The kernel then does what it does
 *            after any timed-out wait: sets bit 0 of q4k_device_error_flags(),
 *            stops waiting, writes no outputs, waits (bounded) for its own
 *            copies in flight and returns; the context stays usable.
 *            Q4K_FLAG_ROWS16: batch 1 on the 16-row-tile kernel (a CTA owns 16
 *            rows over the whole K; its warps split K and add their partial
 *            rows in shared memory, in warp order).  Without the flag the
 *            library takes it by itself for batch 1 when 128-row tiles would
 *            need a K split over CTAs and K <= 8192 (the q/k/v and o
 *            projections of a 7B-class layer); a forced split_k keeps the
 *            128-row kernel.  INVALID_ARG with batch > 1, with
 *            Q4K_FLAG_TENSOR_CORE or with K > 8192.
 *   wait_limit_us  bound of each wait inside the kernel in microseconds;
 *            0 = the default of 2 s.
 */
#define Q4K_FLAG_PDL 1u
#define Q4K_FLAG_TENSOR_CORE 2u
#define Q4K_FLAG_Q8K_X 4u
#define Q4K_FLAG_TEST_STALL 8u
#define Q4K_FLAG_ROWS16 16u
typedef struct {
    int split_k;
    unsigned flags;
    unsigned wait_limit_us;
    int reserved[5];
} q4k_launch_opts;

q4k_status q4k_gemv_ex(const void *W, const float *x, float *y, int64_t N, int64_t K, int batch,
                       void *stream, const q4k_launch_opts *opts);

/*
 * Fused dispatch: up to 4 matrices that multiply the same x (the q/k/v
 * projections of a layer, or its gate/up pair) in one launch, each with its
 * own output.  Same numbers as calling q4k_gemv per matrix with the same
 * split (the row tiles of all matrices share one grid, so the automatic split
 * may differ from the per-matrix one).  The dotLLM README lists this fusion
 * for its CPU decode (News 2026-03 "Fused decode dispatch": Q/K/V 3->1,
 * Gate/Up 2->1).
 *   groups[g].W  Q4_K [N_g][K/256*144] (16-byte aligned), groups[g].y fp32
 *   [batch][N_g]; every matrix has the same K; 1 <= ngroups <= 4; opts may be
 *   NULL.  A matrix with N_g == 0 is skipped.
 */
typedef struct {
    const void *W;
    float *y;
    int64_t N;
} q4k_gemv_group;

q4k_status q4k_gemv_grouped(const q4k_gemv_group *groups, int ngroups, const float *x, int64_t K,
                            int batch, void *stream, const q4k_launch_opts *opts);

/*
 * Read-only streaming probe (a measurement aid; no counterpart on the pages):
 * streams the first *bytes_read bytes of buf from device memory into shared
 * memory the way the GEMV kernels stream their weights -- one CTA per SM,
 * each reading a contiguous slice with 32 KB bulk asynchronous copies through
 * a 4-deep ring -- and discards them.  Timing it gives the read-only HBM rate
 * that bounds the GEMVs (a copy's read+write rate is lower).  *bytes_read is
 * bytes rounded down to a whole number of 32 KB chunks per SM (0 when bytes
 * is smaller).  buf: device pointer, 16-byte aligned; asynchronous on stream.
 * Errors: INVALID_ARG (bytes < 0, null buf or bytes_read), MISALIGNED,
 * UNSUPPORTED_DEVICE, CUDA.
 */
q4k_status q4k_stream_read(const void *buf, int64_t bytes, int64_t *bytes_read, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Rotary positions, the paged cache and attention over it: what stands between
 * a layer's q/k/v products and its output product.
 * ---------------------------------------------------------------------------
 * Tokens are rows of a [tokens][heads][dim] tensor of type Q4K_F32, Q4K_F16 or
 * Q4K_BF16; token and head strides are free (in elements), dim is contiguous.
 *
 * A paged cache holds keys and values in pages of page_size slots each, element
 * (page, slot, head, d) at page*page_stride + slot*slot_stride + head*head_stride
 * + d, for the keys and for the values with strides of their own: page-by-page
 * [slot][head] and [head][slot] orders and keys and values in one buffer are all
 * strides (one of an axis of a single element is not looked at).  Cached
 * position j of sequence b is slot j % page_size of page
 * page_table[b*page_table_stride + j / page_size].  Sequence b of `batch` owns
 * the token rows seq_start[b] .. seq_start[b+1]-1 of the call (none is fine) and
 * kv_len[b] cached positions, these new tokens included: its token i is at
 * position kv_len[b] - (seq_start[b+1] - seq_start[b]) + i.
 *
 * page_table, seq_start, kv_len and the other index arrays are device memory and
 * are read only by the kernels, so a call needs no host copy of them and can be
 * captured in a graph, a process's first one too.  The kernels check them: a
 * position, page, row range or length outside the buffers is not followed (nothing
 * is read or written through it), sets bit 2 of q4k_device_error_flags(), and
 * leaves the outputs that depend on it invalid.  Token rows that belong to no
 * sequence are left as they are.
 *
 * Q4K_FLAG_PDL in a call's flags launches its (first) kernel as a programmatic
 * dependent of the kernel before it on the stream: it may start while that one
 * still runs and waits for its end before it reads anything.
 */
#define Q4K_F32 0
#define Q4K_F16 1
#define Q4K_BF16 2

/* Frequency scaling of q4k_rope_table. */
#define Q4K_ROPE_PLAIN 0  /* f_i = base^(-2i/rot)                                        */
#define Q4K_ROPE_LINEAR 1 /* f_i / factor (positions interpolated)                       */
#define Q4K_ROPE_BASE 2   /* base * factor^(rot/(rot-2)) in place of base                */
#define Q4K_ROPE_RAMP 3   /* f_i / factor for slow pairs, f_i for fast ones, a linear ramp
                             between the pairs that turn `low` and `high` times over
                             orig_len positions (Peng et al., YaRN, 2023)               */
#define Q4K_ROPE_BANDS 4  /* by wavelength w_i = 2 pi / f_i: f_i where w_i < orig_len/high,
                             f_i / factor where w_i > orig_len/low, between them
                             (1-s) f_i / factor + s f_i, s = (orig_len/w_i - low)/(high - low) */

typedef struct {
    double base;      /* > 0, usually 10000 or more */
    double factor;    /* > 0; 1 leaves the frequencies as they are */
    double orig_len;  /* RAMP and BANDS: the context length the model was trained on */
    double low, high; /* RAMP: turns (usually 1 and 32); BANDS: usually 1 and 4; high > low > 0 */
    double magnitude; /* factor on every cosine and sine (RAMP models use 0.1 ln(factor) + 1), usually 1 */
    int32_t scaling;  /* Q4K_ROPE_* */
    int32_t reserved;
} q4k_rope_scaling;

/*
 * table[p][i] = magnitude * cos(p f_i), table[p][rot/2 + i] = magnitude * sin(p f_i)
 * for p < rows, i < rot/2: fp32 [rows][rot], angles and functions formed in fp64
 * (an fp32 angle would be off by 2^-24 p).  Made once, kept by the caller.
 * rows >= 0 (0: no-op), rot even, 2 <= rot <= 512.  Errors: INVALID_ARG,
 * UNSUPPORTED_DEVICE, CUDA.
 */
q4k_status q4k_rope_table(float *table, int64_t rows, int64_t rot, const q4k_rope_scaling *s, void *stream);

/*
 * y = x with each head turned by its token's table row: for i < rot/2 the pair
 * (a, b) = (x[i], x[i + rot/2]), or (x[2i], x[2i+1]) with `interleaved`, becomes
 * (a c - b s, a s + b c); elements rot .. dim-1 are copied.  Arithmetic in fp32,
 * one rounding to y's type.  Token t uses row pos[t].  y may be x itself (same
 * type and strides); they must not overlap otherwise.
 *   tokens >= 0 (0: no-op), heads >= 1, dim >= 1, rot even, 0 <= rot <= dim and
 *   <= 512 (rot = 0 copies; pos and table may then be NULL); any alignment of
 *   the element type (16-byte aligned rows take wide loads).
 * Errors: INVALID_ARG, MISALIGNED (a pointer not aligned to its element),
 * UNSUPPORTED_DEVICE, CUDA.
 */
typedef struct {
    const void *x;
    void *y;
    const int32_t *pos; /* [tokens] */
    const float *table; /* [table_rows][rot] */
    int64_t tokens, heads, dim, rot, table_rows;
    int64_t x_token_stride, x_head_stride, y_token_stride, y_head_stride;
    int32_t x_type, y_type, interleaved;
    uint32_t flags; /* Q4K_FLAG_PDL or 0 */
} q4k_rope_args;

q4k_status q4k_rope(const q4k_rope_args *a, void *stream);

typedef struct {
    void *k, *v;
    int64_t k_page_stride, k_slot_stride, k_head_stride;
    int64_t v_page_stride, v_slot_stride, v_head_stride;
    int64_t pages, page_size, heads, dim;
    const int32_t *page_table; /* [batch][page_table_stride], max_pages of each row used */
    int64_t page_table_stride, max_pages;
    const int32_t *seq_start; /* [batch + 1] */
    const int32_t *kv_len;    /* [batch] */
    int64_t batch, tokens;
    int32_t type;             /* Q4K_F16 or Q4K_BF16 */
    int32_t reserved;
} q4k_paged_cache;

/*
 * Stores the new tokens' keys and values in the cache, the keys turned as
 * q4k_rope turns them (row pos[t], or the token's cache position where pos is
 * NULL), and turns the queries into q_out in the same launch where q is given.
 * Rounding: fp32 arithmetic, then once to the cache's (q_out's) type.
 *   k, v [tokens][cache heads][dim] of type kv_type; q, q_out
 *   [tokens][q_heads][dim] (NULL: none); rot = 0: nothing is turned (table NULL).
 *   The slots written must be distinct over the call; q_out may be q itself.
 * Only the new tokens' slots of the cache are written.
 * Errors: as q4k_rope.
 */
typedef struct {
    const void *k, *v, *q;
    void *q_out;
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    int64_t q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride;
    const int32_t *pos;
    const float *table;
    int64_t table_rows, rot, q_heads;
    int32_t kv_type, q_type, q_out_type, interleaved;
    uint32_t flags; /* Q4K_FLAG_PDL or 0 */
    int32_t reserved;
} q4k_append_args;

q4k_status q4k_kv_append(const q4k_paged_cache *c, const q4k_append_args *a, void *stream);

/*
 * Attention of the new tokens (one or many per sequence) over the paged cache.
 * Query head h reads cache head h / (q_heads / cache heads).  Token t at
 * position p of sequence b sees the positions lo <= j < hi with
 *   hi = kv_len[b] without `causal`, else min(kv_len[b], max(p + 1, prefix_len[b])),
 *   lo = max(0, kv_start[t], p + 1 - window)
 * (prefix_len, kv_start NULL and window 0: not applied) and gets
 *   s_j = scale q.k_j,  s_j = softcap tanh(s_j / softcap) (softcap > 0),
 *   s_j = s_j - slopes[h] |p - j| (slopes not NULL),
 *   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  lse = m + ln sum_j exp(s_j - m).
 * A row that sees nothing, or only scores of -inf, gives out = 0, lse = -inf.
 * Slots that no token of a sequence's query tile sees may hold anything,
 * infinities and NaN included; an infinite or NaN value that some token sees may
 * also reach nearby tokens that do not see it (an infinite one as NaN).
 *
 * Precision: softmax statistics, sums and outputs accumulate in fp32.  With q of
 * the cache's type and a 16-bit out, the weights exp(s_j - m) are rounded once to
 * the cache's type before they meet the values on the tensor cores (each by
 * at most 2^-8 of itself in bf16, 2^-11 in fp16, beside the output's own rounding).
 * With fp32 q or out, q and the weights enter as 2 (fp16) or 3
 * (bf16) parts, 22 and 24 bits; so they do with a softcap above 256, whose scores
 * are formed to 2^-20 of themselves (2^-22 of the cap below that, in 16-bit calls).
 * A softcap above 1e30 is taken as 1e30, one below 1e-30 as that.
 *
 *   q, out [tokens][q_heads][dim]: any type each; lse fp32 [tokens][q_heads] or NULL
 *   q_heads a positive multiple of the cache's heads, dim a multiple of 8,
 *   8 <= dim <= 256; 16-byte aligned k, v, q, out and strides that keep every
 *   row 16-byte aligned; tokens * q_heads < 2^31.
 *   causal 0 or 1; window >= 0; softcap >= 0 and finite.
 * Calls that split rows over the whole GPU (a few long sequences, prompt chunks)
 * take scratch on `stream` from a stream-ordered pool of the library's own, which
 * keeps it for later calls (to the end of the process): for each call in flight at
 * most 8 R (W + 2) bytes an SM, R the rows of its tiles, W dim rounded up to 64,
 * 128 or 256; on 152 SMs 0.6 MB (8 rows of 64) to 40.5 MB (256 rows of 128).
 * Partial results are added in a fixed order: the same inputs give the same bits.
 * Q4K_FLAG_TEST_STALL makes a CTA's first copies be awaited for 16 bytes more than
 * they bring (where pages hold a multiple of 16 slots); the kernel then winds down
 * as after any wait that runs out (bit 3 of the error flags, outputs invalid).
 * Q4K_FLAG_ATTN_FORM(n) has a call take one form of the kernels, normally chosen
 * by the library from the sizes: tiles of 8, 16 or 32 query rows, each by a cluster
 * of CTAs (Q4K_ATTN_CLUSTER8, 16, 32) or with the work split over the GPU
 * (Q4K_ATTN_SPLIT8, 16, 32; tiles of 32 for dim <= 128), or tiles of 256 rows on
 * tcgen05 (Q4K_ATTN_MANY: q of the cache's type, a 16-bit out, dim <= 128, pages of
 * a multiple of 16, scale >= 0, softcap <= 256); INVALID_ARG where the call cannot take it.  Errors: INVALID_ARG, MISALIGNED, UNSUPPORTED_DEVICE, CUDA.
 */
typedef struct {
    const void *q;
    void *out;
    float *lse;
    int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
    int64_t q_heads, window;
    const float *slopes;       /* [q_heads] or NULL */
    const int32_t *prefix_len; /* [batch] or NULL */
    const int32_t *kv_start;   /* [tokens] or NULL */
    float scale, softcap;
    int32_t q_type, out_type, causal;
    uint32_t flags;         /* Q4K_FLAG_PDL, Q4K_FLAG_TEST_STALL (failure-path tests only), Q4K_FLAG_ATTN_FORM(n) or 0 */
    uint32_t wait_limit_us; /* bound of each wait inside the kernel; 0 = 2 s (when one runs out, what is in flight
                               is awaited, 20 ms at most each) */
    int32_t reserved;
} q4k_attention_args;

#define Q4K_FLAG_ATTN_FORM(n) ((uint32_t)(n) << 8)
#define Q4K_ATTN_CLUSTER8 1
#define Q4K_ATTN_CLUSTER16 2
#define Q4K_ATTN_CLUSTER32 3
#define Q4K_ATTN_SPLIT8 4
#define Q4K_ATTN_SPLIT16 5
#define Q4K_ATTN_SPLIT32 6
#define Q4K_ATTN_MANY 7

q4k_status q4k_paged_attention(const q4k_paged_cache *c, const q4k_attention_args *a, void *stream);

/*
 * ---------------------------------------------------------------------------
 * The paged cache in 8 bits: codes with a scale for each block of tokens and
 * head.  Half the memory of a 16-bit cache, half the bytes of a decode step.
 * ---------------------------------------------------------------------------
 * Codes lie in pages as in q4k_paged_cache (whose strides count elements, here
 * bytes), of type Q4K_I8 (-127 .. 127) or Q4K_E4M3 (4 exponent and 3 fraction
 * bits, up to 448).  The slots of a page are cut into blocks of `block`
 * consecutive ones, and each block has one fp32 scale per head, for the keys and
 * for the values: the value of (page, slot, head, d) is its code times the scale at
 * page*page_stride + (slot / block)*block_stride + head*head_stride.  A block of one
 * token costs 4 bytes a head and token and is never scaled anew; larger ones cost less
 * and share their largest value.
 */
#define Q4K_I8 3
#define Q4K_E4M3 4

typedef struct {
    q4k_paged_cache cache; /* type: Q4K_I8 or Q4K_E4M3 */
    float *k_scale, *v_scale;
    int64_t k_scale_page_stride, k_scale_block_stride, k_scale_head_stride;
    int64_t v_scale_page_stride, v_scale_block_stride, v_scale_head_stride;
    int64_t block; /* a power of two up to 128 that divides page_size */
} q4k_paged_cache8;

/*
 * y = turn(x * weight / sqrt(mean(x^2) + eps)) for the heads of one or two tensors
 * (queries and keys) in one launch: the mean over a head's dim elements, the rotation
 * as q4k_rope's (row pos[t] of the table).  fp32 arithmetic, one rounding to y's type.
 *   weight fp32 [dim], or [heads][dim] with weight_head_stride = dim; NULL: that
 *   tensor is not normed.  k.x NULL: one tensor.  y may be x itself (same type and
 *   strides); the tensors must not overlap otherwise.
 *   tokens >= 0 (0: no-op), dim a multiple of 8 up to 256, rot even, 0 <= rot <= dim
 *   (0: nothing is turned; pos and table may then be NULL), eps >= 0 and finite.
 * Errors: as q4k_rope.
 */
typedef struct {
    const void *x;
    void *y;
    const float *weight;
    int64_t heads, x_token_stride, x_head_stride, y_token_stride, y_head_stride, weight_head_stride;
    int32_t x_type, y_type;
} q4k_heads;

typedef struct {
    q4k_heads q, k;
    const int32_t *pos; /* [tokens] */
    const float *table; /* [table_rows][rot] */
    int64_t tokens, dim, rot, table_rows;
    float eps;
    int32_t interleaved;
    uint32_t flags; /* Q4K_FLAG_PDL or 0 */
    int32_t reserved;
} q4k_norm_rope_args;

q4k_status q4k_norm_rope(const q4k_norm_rope_args *a, void *stream);

/*
 * q4k_kv_append into an 8-bit cache: keys normed (k_weight, NULL: not) and turned,
 * values as they come, both in fp32; queries, where given, normed (q_weight) and
 * turned into q_out.  With top = 127 or 448, a block that new tokens fall into gets
 *   scale = max(max|x| / top over its new tokens, its old |scale| where it holds older
 *           tokens of the sequence (positions before the first new one), 2^-126),
 *   code = x * (1 / scale) rounded to nearest even, at most top in size,
 * and where that scale has changed the older tokens' codes become code * (old scale / scale),
 * rounded again (by at most half a step of the new scale).  Slots behind the first new
 * position count as empty: what an engine takes back is not asked.  Infinities do not
 * count for the scale and are stored as +-top; a NaN is stored as 0 (Q4K_I8) or NaN
 * (Q4K_E4M3).  Only the new tokens' slots, the older ones of their blocks and those
 * blocks' scales are written; a block that new tokens fall into belongs to one sequence
 * of the call.  dim a multiple of 8 up to 256; no stride of the cache or its scales is 0
 * along an axis of more than one (INVALID_ARG); everything else as q4k_kv_append.
 */
typedef struct {
    q4k_append_args a;
    const float *q_weight, *k_weight; /* as in q4k_heads */
    int64_t q_weight_head_stride, k_weight_head_stride;
    float eps;
    int32_t reserved;
} q4k_append8_args;

q4k_status q4k_kv_append8(const q4k_paged_cache8 *c, const q4k_append8_args *a, void *stream);

/*
 * Reads cached rows back: token row t of sequence b gets scale * code of its position
 * (the positions that q4k_kv_append8 with the same arrays writes; for whole sequences
 * seq_start counts up kv_len), formed in fp32 and rounded once to `type` (Q4K_F32,
 * Q4K_F16 or Q4K_BF16).
 *   k, v [tokens][heads][dim]; either may be NULL.  Rows of no sequence and rows whose
 *   position or page is outside the buffers are left as they are (the latter set bit 2
 *   of the error flags).  dim a multiple of 8 up to 256.  Errors: as q4k_rope.
 */
typedef struct {
    void *k, *v;
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    int32_t type;
    uint32_t flags; /* Q4K_FLAG_PDL or 0 */
} q4k_read8_args;

q4k_status q4k_kv_read8(const q4k_paged_cache8 *c, const q4k_read8_args *a, void *stream);

/*
 * q4k_paged_attention over an 8-bit cache: the same masks, scores and outputs, with
 * scale * code for every key and value.  The codes are multiplied as they are (exact
 * in fp16); keys' scales enter the scores, values' the softmax weights, in fp32.
 * Precision: with 16-bit q and out, q enters as fp16 over a power of two per row (bf16
 * values below 2^-38 of the row's largest lose bits) and the weights, with their
 * values' scales, are rounded once to fp16 (2^-11 at most); with fp32 q or out, or a
 * softcap above 256, both enter as two fp16 parts (22 bits).  A weight times its value's
 * scale counts to 2^-38 of the largest scale of the values that its tile meets (2^-29 in
 * the many-rows form).  The rest is in fp32.
 * The many-rows form (prompt chunks; fp16 or bf16 q and out, dim up to 128, pages of a
 * multiple of 16 slots) turns the codes into fp16 scratch first.  With blocks of 16 tokens
 * or more they stay exact; with smaller ones scale * code, over a power of two for each 16
 * tokens, is rounded once to fp16 (2^-11, or 2^-31 of the largest scale of those of the 16
 * that the sequence's tokens see).  It takes 4 * dim bytes of stream-ordered scratch
 * a table position of each sequence and cache head, up to 4 GiB; past that heads, then
 * sequences go through in passes, and where one head of one sequence has no room the call
 * takes another form (asked for by name it is refused).  (Where the device has less to
 * give the passes get smaller.)  bf16 queries come on top: 2 * dim + 4 bytes a token and
 * query head of a pass.  That scratch is a call's in flight and the page table's width
 * sets it, not the lengths; its memory stays with the library as q4k_scratch_keep says.
 * Slots that no token of a sequence's query tile sees may hold anything, their scales
 * too.  A block whose scale a token sees must have one that is finite: NaN makes the
 * token's rows NaN, and may those of nearby tokens.
 *   dim a multiple of 16 up to 256; k and v 16-byte aligned, with strides that keep
 *   every row 16-byte aligned; everything else as q4k_paged_attention.
 */
q4k_status q4k_paged_attention8(const q4k_paged_cache8 *c, const q4k_attention_args *a, void *stream);

/*
 * How much free memory the current device's pool of that scratch may hold when the program
 * synchronises (a stream, an event or the device); the rest goes back to the system.  It
 * has a pool of its own beside q4k_paged_attention's, with 5 GiB to begin with.  0: all of
 * it goes back each time, and the first call after that waits for it (0.7 ms a GiB).  A
 * captured call's scratch belongs to its graph.  bytes >= 0, else INVALID_ARG.
 */
q4k_status q4k_scratch_keep(int64_t bytes);

/* Launch plan the automatic heuristics pick for a shape (for tests and
 * reports): out[0] = split_k, out[1] = number of CTAs, out[2] = rows per CTA
 * tile, out[3] = K blocks per x chunk held in shared memory. */
q4k_status q4k_gemv_plan(int64_t N, int64_t K, int batch, int out[4]);

/* Sticky device-side error bits of the library's kernels, read synchronously
 * from the current device: bit 0 = a bounded wait inside a GEMV/argmax
 * kernel (Q4_K or Q6_K) or the streaming probe timed out, bit 1 = the same in the prefill
 * kernel; the kernel then wound down early and its outputs are invalid;
 * bit 2 = an index array of q4k_rope, q4k_norm_rope, q4k_kv_append(8), q4k_kv_read8
 * or q4k_paged_attention(8) points outside its buffers; bit 3 = a bounded wait in q4k_paged_attention(8).
 * 0 = no error.  The bits stay set until q4k_device_error_clear(). */
unsigned int q4k_device_error_flags(void);

/* Reset the sticky error bits on the current device (synchronous; call it
 * when no kernel of the library is running).  Q4K_ERR_CUDA if a copy to the
 * device failed. */
q4k_status q4k_device_error_clear(void);

#ifdef __cplusplus
}
#endif

#endif /* Q4K_H */
