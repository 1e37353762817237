/*
 * kvr.h - C ABI of libkvr.so, the GB300 (sm_103a) attention-prologue key path.
 *
 * The operations:
 *
 *   kv_rmsnorm_rope_cache()  the fused KV prologue of the page
 *       "aclnnKvRmsNormRopeCache" (hiascend.com, CANN ops-transformer):
 *       each token row of width D = Dv + Dk is split on its tail axis
 *       ("Description"); the left Dv part is RMS-normalised
 *       ("Formulas (2) rmsNorm": y = x / sqrt(mean(x^2) + eps) * gamma),
 *       the right Dk part gets the interleaved RoPE ("Formulas (1)
 *       interleaveRope": y = cat(x[::2], x[1::2]) * cos + cat(-x[1::2], x[::2]) * sin),
 *       and both results are scattered by slot index into two caches
 *       ("Restrictions on index"), optionally quantised to 8-bit codes
 *       ("Restrictions on quantization scenarios"). The kcScale factor
 *       alpha_kv of "aclnnMlaPrologV3WeightNz" ("Formula", key path) may
 *       scale the normalised part.
 *
 *   qsa_prepare()  the block-key prepare of "openvino.opset17.qsa_prepare"
 *       (docs.openvino.ai): one key per key block completed by the new
 *       tokens = mean of the block's raw index keys, RMS-normalised with
 *       k_norm_weight, rotated with the RoPE of the block's first token;
 *       incomplete blocks are carried across calls.
 *
 *   dynamic_quant()  DynamicQuant of q^N, the query-side step beside this
 *       path on "aclnnMlaPrologV3WeightNz": per-row int8 codes and scales.
 *
 *   query_rope()  the rotary positions of the query's rotary part q^R, with one
 *       position per axis (time, height, width, ...); it can write the cos/sin
 *       tables that kv_rmsnorm_rope_cache() takes for the same tokens.
 *
 *   mla_attention()  attention of new tokens (one per sequence, a few, or a
 *       chunk) over the caches kv_rmsnorm_rope_cache() fills: every head reads
 *       the same latent row as key and as value.
 *
 *   kv_cache_read()  the cache rows of an index read back into dense rows,
 *       8-bit codes decoded.
 *
 *   draft_tree(), mla_tree_attention()  a tree of drafted tokens: the ancestors
 *       and the positions of its tokens, and mla_attention() where each of them
 *       sees its ancestors.
 *
 *   mla_key_weight(), kv_cache_select(), kv_cache_compact()  caches of bounded
 *       size: the attention weight that each key receives, the keys to keep by
 *       it, and kept rows moved together (an accepted branch of a tree too).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller (the
 *     host-staged entry points also take pinned host buffers); the library
 *     allocates no device memory and keeps no per-call state, with one
 *     exception: kv_rmsnorm_rope_cache_staged_static stages its inputs in a
 *     static device array of the library, shared by all its calls on a
 *     device. Rows are dense and row-major unless a stride argument says
 *     otherwise.
 *   - Calls are asynchronous on `stream`: they validate on the host, launch,
 *     and return. Nothing is read back to the host (except the status word
 *     the host-staged entry point copies back, asynchronously, and the index
 *     that the opt-in debug validation, kvr_set_debug_validate, checks).
 *   - Host-side errors (a NULL that is required, a bad shape, dtype or
 *     mode) are returned before any launch; nothing is written. Sizes whose
 *     element offsets or byte counts would reach 2^62 are KVR_ERR_SHAPE.
 *   - Data-dependent errors are found on the device: the offending row or
 *     block is skipped (never written out of bounds) and, if `dev_status`
 *     is non-NULL, the matching KVR_DEVERR_* bit is OR-ed into *dev_status.
 *     No kernel traps or asserts. Waits inside a kernel (its copy pipeline)
 *     are bounded: past one second a kernel raises KVR_DEVERR_TIMEOUT, lets
 *     its copies in flight land, and returns.
 *   - Each launch uses programmatic dependent launch: it may start while the
 *     previous kernel on the stream finishes, and waits for that kernel's
 *     results before it uses any input (the one exception is opt-in:
 *     the params_ready flags let constants be read earlier). Before the wait
 *     a kernel issues L2 prefetches of its inputs; qsa_prepare's
 *     compiled-shape kernel also reads key_length there, as a hint for those
 *     prefetches only (a relaxed read; kvr_qsa_args.key_length_late turns
 *     it off), and takes its value after the wait.
 *   - An empty problem (T = Bkv*Skv = 0, or N = 0) returns KVR_OK with no
 *     launch, mirroring the empty-tensor rule of "aclnnMlaPrologV3WeightNz"
 *     ("Shape restrictions": caches are not updated). A qsa_prepare call
 *     with L = 0 launches only when it has carry outputs or a separate past
 *     buffer to write.
 *   - Results are deterministic: no atomics touch data.
 *   - Thread safe: entry points may be called concurrently from any host
 *     thread on any stream; overlapping writes to the same cache rows from
 *     concurrent calls are the caller's race. The exception is
 *     kv_rmsnorm_rope_cache_staged_static: its calls that can run at the
 *     same time on the GPU share its staging area and race on it.
 */
#ifndef KVR_H
#define KVR_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KVR_ABI_VERSION 10

typedef enum kvr_status {
    KVR_OK = 0,
    KVR_ERR_NULL = 1,         /* a required pointer is NULL, or optional pairs disagree */
    KVR_ERR_SHAPE = 2,        /* a size is out of its documented range */
    KVR_ERR_DTYPE = 3,        /* an element type is not supported for that argument */
    KVR_ERR_MODE = 4,         /* unknown cache mode */
    KVR_ERR_ALIAS = 5,        /* an output overlaps an input it must not overlap */
    KVR_ERR_CUDA = 6,         /* the launch failed (see cudaGetLastError) */
    KVR_ERR_INDEX = 7         /* debug validation only (kvr_set_debug_validate): an index
                                 entry is out of range or names a cache row that another
                                 entry of the call names */
} kvr_status;

/* Bits OR-ed into *dev_status by the kernels. */
#define KVR_DEVERR_INDEX 0x1       /* kv, read: an index entry outside {-1} U [0, range); attention, key
                                      weight: such an entry of the block table that a token sees; tree:
                                      a parent that does not come before; compact: a kept entry out of
                                      order or a row that cannot be moved */
#define KVR_DEVERR_KEY_LENGTH 0x2  /* qsa: key_length[n] < L (the past length would be negative);
                                      attention, key weight, select, compact: a length that is negative
                                      or beyond what there is room for */
#define KVR_DEVERR_BLOCK_CAP 0x4   /* qsa: a completed block's number is >= Bcap */
#define KVR_DEVERR_TIMEOUT 0x8     /* a pipeline wait inside a kernel exceeded its limit (one second, in
                                      mla_attention and one more for 2^22 keys of a part before, in
                                      mla_key_weight for 2^22 rows of queries and for 2^22 keys that
                                      there is room for); that CTA stopped early, output incomplete */
#define KVR_DEVERR_PAST_BLOCKS 0x10 /* qsa, concat-output form: past_block_index_keys holds
                                      fewer than floor(P/kbs) rows for a sequence */
#define KVR_DEVERR_QUERY 0x20      /* attention, key weight, tree: query_start decreases or leaves [0, T]
                                      at a sequence, or it has more tokens than tree_mask has bits */

typedef enum kvr_dtype {
    KVR_BF16 = 0,
    KVR_F16 = 1,
    KVR_INT8 = 2,             /* caches only: round half to even, clamp to [-128, 127] */
    KVR_FP8_E4M3FN = 3,       /* caches only: round to nearest even, saturate to +-448 */
    KVR_FP8_E5M2 = 4          /* caches only: round to nearest even, saturate to +-57344 */
} kvr_dtype;

/* Cache layouts of "aclnnKvRmsNormRopeCache" ("Restrictions on index"); the
 * head axis N is 1, so BNSD and BSND are the same bytes. */
typedef enum kvr_cache_mode {
    /* cache [Bcache=d0, Scache=d1, 1, D*]; index [Bkv, Skv] in [-1, Scache);
     * token (b, s) goes to cache row (b, index[b, s]); requires Bcache >= Bkv. */
    KVR_CACHE_NORM = 0,
    /* cache [BlockNum=d0, BlockSize=d1, 1, D*]; index [Bkv*Skv] in
     * [-1, BlockNum*BlockSize); token t goes to slot index[t]. */
    KVR_CACHE_PA_BSND = 1,
    /* cache as PA_BSND; index [Bkv * ceil(Skv/BlockSize)], one entry per
     * BlockSize tokens of a sequence; token s goes to slot
     * index[b, s / BlockSize] + s % BlockSize, which must stay inside the
     * block the entry names (else KVR_DEVERR_INDEX). */
    KVR_CACHE_PA_BLK_BSND = 2
} kvr_cache_mode;

/*
 * Arguments of kv_rmsnorm_rope_cache(). T = Bkv * Skv token rows.
 *
 *   kv         [Bkv, 1, Skv, >= Dv+Dk] input rows, element type `in_dtype`
 *              (bf16 or f16). Row t starts kv_row_stride elements after row
 *              t-1 (0 means Dv+Dk, i.e. dense); a larger stride reads kv as
 *              a column slice of a wider row (e.g. a fused projection output).
 *   gamma      [Dv] RMSNorm weight, `in_dtype`.
 *   cos, sin   [Bkv, 1, Skv, Dk] full-width RoPE tables, `in_dtype`; output
 *              lane i < Dk/2 uses entry i, lane i + Dk/2 uses entry i + Dk/2.
 *   index      int64, layout per `mode` (see kvr_cache_mode); -1 = skip.
 *              Repeated targets within one call (forbidden by the page) leave
 *              an unspecified winner.
 *   cache_d0, cache_d1   the two leading cache dims (Bcache, Scache) or
 *              (BlockNum, BlockSize).
 *   ckv_cache  [d0, d1, 1, Dv] of `ckv_dtype`; k_cache [d0, d1, 1, Dk] of `k_dtype`.
 *              A cache dtype is `in_dtype` (bf16/f16) or an 8-bit code type.
 *   ckv_scale  float32 [ckv_scale_len], len Dv (per channel) or 1 (per
 *              tensor); required iff ckv_dtype is an 8-bit type, else NULL.
 *              The code written is encode(alpha_kv * y[c] * ckv_scale[c]).
 *   k_scale    same for the k cache (len Dk or 1), applied to the RoPE output lane c.
 *   eps        added to the mean square (>= 0).
 *   kc_scale   alpha_kv, multiplies the normalised part; pass 1.0f for none.
 *   dev_status optional int32 device word; KVR_DEVERR_INDEX is OR-ed in when
 *              an index entry is out of range (that token is skipped).
 *   params_ready  0 (default): every input is read after the kernel waits for
 *              the preceding kernel on the stream (programmatic dependent
 *              launch). Nonzero: the caller promises that the kernel launched
 *              immediately before this call on `stream` does not write gamma,
 *              ckv_scale or k_scale (true of model weights and calibrated
 *              scales); they may then be read before that wait, overlapping
 *              the preceding kernel (the small-batch kernel for 16-bit caches
 *              does not, as that measured slower). Breaking the promise gives
 *              stale values.
 *
 * Limits: Dv >= 1, Dk >= 2 and even, Bkv, Skv >= 0, d0, d1 >= 1.
 * All arithmetic is float32 with one rounding to the cache type.
 */
typedef struct kvr_kv_args {
    const void* kv;
    kvr_dtype in_dtype;
    int64_t Bkv, Skv, Dv, Dk;
    int64_t kv_row_stride;
    const void* gamma;
    const void* cos;
    const void* sin;
    const int64_t* index;
    kvr_cache_mode mode;
    int64_t cache_d0, cache_d1;
    void* ckv_cache;
    kvr_dtype ckv_dtype;
    const float* ckv_scale;
    int64_t ckv_scale_len;
    void* k_cache;
    kvr_dtype k_dtype;
    const float* k_scale;
    int64_t k_scale_len;
    float eps;
    float kc_scale;
    int32_t* dev_status;
    int32_t params_ready;
} kvr_kv_args;

kvr_status kv_rmsnorm_rope_cache(const kvr_kv_args* args, cudaStream_t stream);

/*
 * Host-staged form of kv_rmsnorm_rope_cache (no counterpart on the pages: a
 * convenience for callers whose inputs are in host memory). On `stream`, in
 * order: copy `bytes` bytes from host memory `host_src` to device memory
 * `dev_dst` (the caller lays the step's inputs out there, so that the device
 * pointers in *args point into it), run kv_rmsnorm_rope_cache(args), and,
 * when `host_status` is given, copy *args->dev_status into *host_status.
 * All asynchronous: the host values are read and written when the stream
 * reaches the copies, so `host_src` and `host_status` should be pinned
 * (page-locked) and stay valid until the stream passes them; the caller
 * synchronises before reading *host_status. Arguments are validated first
 * and nothing is enqueued on an error (as kv_rmsnorm_rope_cache; plus
 * KVR_ERR_SHAPE for bytes < 0, KVR_ERR_NULL for a missing copy pointer or a
 * host_status without args->dev_status). A failed enqueue returns
 * KVR_ERR_CUDA (copies enqueued before it stay enqueued). Pinned buffers
 * (reported as host memory with a device address) in whole 16-byte units
 * are copied by kernels chained with the call (no copy-engine latency);
 * other memory goes through cudaMemcpyAsync.
 */
kvr_status kv_rmsnorm_rope_cache_staged(const kvr_kv_args* args, const void* host_src, void* dev_dst, int64_t bytes,
                                        int32_t* host_status, cudaStream_t stream);

/* Largest packed input, in bytes, that kv_rmsnorm_rope_cache_staged_static
 * stages: 8 MiB (a 256-token decode batch of the 512 + 64 split packs into
 * 354 KiB, a 4096-token batch into 5.5 MiB). */
#define KVR_STATIC_STAGE_BYTES (8 * 1024 * 1024)

/*
 * kv_rmsnorm_rope_cache_staged for callers that cannot allocate device memory
 * (no counterpart on the pages). The host-staged call needs a device buffer
 * to copy the step's inputs into, and some callers have none to give: code
 * running where cudaMalloc is not allowed (inside an allocator's own
 * callbacks, or under a framework that owns all device memory and offers its
 * plugins no way to ask for more) or a process whose memory budget is spent.
 * This entry point allocates nothing: it stages into one area of
 * KVR_STATIC_STAGE_BYTES that the library holds as a static device array on
 * every device that loads it, from load until the process exits.
 *
 *   args        as for kv_rmsnorm_rope_cache, except that args->kv, cos, sin
 *               and index are ignored: those four inputs are read from the
 *               staging area at the byte offsets below.
 *   host_src    `bytes` bytes of packed inputs in host memory (pinned for the
 *               copy to run as a kernel, as for kv_rmsnorm_rope_cache_staged);
 *               kv at kv_offset, cos at cos_offset, sin at sin_offset (each a
 *               multiple of 2) and index at index_offset (a multiple of 8),
 *               laid out as kv_rmsnorm_rope_cache expects them.
 *   bytes       at most KVR_STATIC_STAGE_BYTES; every input must lie inside
 *               [0, bytes), so each byte the call reads was written by its own
 *               copy and nothing in the area has to start at zero.
 *   host_status as for kv_rmsnorm_rope_cache_staged.
 *
 * Errors: bytes < 0 or > KVR_STATIC_STAGE_BYTES: KVR_ERR_SHAPE; an input
 * that does not fit inside [0, bytes) at its offset (the T kv rows at their
 * row stride, the cos and sin tables, the index entries of the mode; so in
 * particular a row width or row stride larger than `bytes`) or is misaligned:
 * KVR_ERR_SHAPE; nothing is enqueued on these errors. Everything else as
 * kv_rmsnorm_rope_cache_staged (KVR_ERR_CUDA if the area's address cannot be
 * found). Every call with T > 0 looks up the area's device address in the
 * current context (cudaGetSymbolAddress, which allocates nothing); the first
 * such call on a device may load the library's device code there, so make
 * it before any stream capture on the device. The address is never kept
 * between calls, so a device reset or another context stays safe. All calls
 * on a device share the one area, which keeps the last call's contents:
 * calls on the same stream are ordered, but calls that can run at the same
 * time on the GPU (other streams, other host threads) overwrite each other's
 * inputs.
 */
kvr_status kv_rmsnorm_rope_cache_staged_static(const kvr_kv_args* args, const void* host_src, int64_t bytes,
                                               int64_t kv_offset, int64_t cos_offset, int64_t sin_offset,
                                               int64_t index_offset, int32_t* host_status, cudaStream_t stream);

/* Which Dr channels the QSA rotation acts on and how it pairs them (the
 * qsa_prepare page names neither). Every layout writes pair i's results to
 * lanes i and i + Dr/2 of the rotated channels with cos/sin lanes i and
 * i + Dr/2, as the interleaved RoPE of "aclnnKvRmsNormRopeCache" does. */
typedef enum kvr_qsa_rope {
    KVR_QSA_ROPE_INTERLEAVE_LAST = 0,   /* pairs (x[2i], x[2i+1]) of channels [Di-Dr, Di) */
    KVR_QSA_ROPE_INTERLEAVE_FIRST = 1,  /* the same pairs of channels [0, Dr) */
    KVR_QSA_ROPE_HALF_LAST = 2,         /* rotate-half pairs (x[i], x[i+Dr/2]) of [Di-Dr, Di) */
    KVR_QSA_ROPE_HALF_FIRST = 3         /* rotate-half pairs of [0, Dr) */
} kvr_qsa_rope;

/*
 * Arguments of qsa_prepare(). Inputs follow the parameter list of
 * "openvino.opset17.qsa_prepare".
 *
 *   raw_index_keys  [N, L, Di] raw index key of every new token, `in_dtype`.
 *   block_keys      [N, Bcap, Di] in/out, `in_dtype`: the block keys of
 *                   earlier calls (past_block_index_keys) followed by room for
 *                   new ones. Block j (tokens [j*kbs, (j+1)*kbs) of the
 *                   sequence) is written at row j; no other row is touched.
 *                   In the concat-output form (below) rows j < floor(P/kbs)
 *                   are first copied from past_block_index_keys.
 *   key_length      int64 [N] or [1] (key_length_len = N or 1): valid key
 *                   tokens of each sequence AFTER this call, so the past
 *                   length is P = key_length - L (< 0: KVR_DEVERR_KEY_LENGTH,
 *                   the sequence is skipped). A [1] value applies to all N.
 *   rope_cos, rope_sin  [N, L, Dr] RoPE of every new token, or both NULL to
 *                   disable the rotation. By default the rotation is the
 *                   interleaved RoPE of "aclnnKvRmsNormRopeCache" on channels
 *                   [Di-Dr, Di); rope_layout selects another (kvr_qsa_rope).
 *   k_norm_weight   [Di] or NULL (NULL disables the RMS normalisation).
 *   past_incomplete_raw_keys  [N, kbs-1, Di]: raw keys of the past tokens of
 *                   the incomplete block (rows >= P mod kbs are never read).
 *   past_incomplete_rope      [N, 2*Dr] = [cos | sin] of the incomplete
 *                   block's first token; NULL iff rope_cos is NULL. Read only
 *                   when P mod kbs > 0.
 *   key_block_size  kbs > 1.   eps >= 0.
 *   next_incomplete_raw_keys  optional out [N, kbs-1, Di]: raw keys of the
 *                   tokens after the last completed block (K mod kbs rows;
 *                   the other rows are left untouched).
 *   next_incomplete_rope      optional out [N, 2*Dr]: [cos | sin] of the
 *                   first of those tokens (untouched when K mod kbs = 0).
 *                   The next_* outputs must not overlap any input
 *                   (KVR_ERR_ALIAS), so two carry buffers alternate between calls.
 *   dev_status      optional int32 device word (KVR_DEVERR_KEY_LENGTH,
 *                   KVR_DEVERR_BLOCK_CAP, KVR_DEVERR_PAST_BLOCKS).
 *   rope_layout     kvr_qsa_rope (0, the default, keeps the reading above).
 *   past_block_index_keys, Bp  concat-output form: [N, Bp, Di] `in_dtype`,
 *                   the page's past_block_index_keys as a separate input.
 *                   NULL (or equal to block_keys) = in place: block_keys
 *                   already holds them. Otherwise rows j < min(Bp,
 *                   floor(P/kbs)) are copied to block_keys (past rows at or
 *                   beyond Bcap: KVR_DEVERR_BLOCK_CAP; Bp < floor(P/kbs):
 *                   KVR_DEVERR_PAST_BLOCKS, the missing rows stay untouched),
 *                   so block_keys ends as the past keys followed by the new
 *                   ones. It must not overlap block_keys or the next_* outputs.
 *   params_ready    0 (default): every input is used as read after the kernel
 *                   waits for the preceding kernel on the stream (programmatic
 *                   dependent launch); the compiled-shape kernel reads
 *                   key_length once before that wait as a prefetch hint and
 *                   compares it with the value read after it (a stale hint,
 *                   e.g. key_length written by that preceding kernel, costs
 *                   time, never correctness: the warp sums its block a second
 *                   time, about 2 us on the 32 x 2048-token workload). Nonzero:
 *                   the caller promises that the
 *                   kernel launched immediately before this call on `stream`
 *                   writes none of key_length, rope_cos, rope_sin,
 *                   past_incomplete_rope and k_norm_weight (true when
 *                   sequence lengths come from the scheduler, the tables are
 *                   precomputed and the weight is a model weight); the kernel
 *                   for the compiled shapes (Di in {64, 128, 256}, kbs in
 *                   {32, 64, 128}, 16-byte aligned) then reads them before
 *                   that wait, so that only the key rows are read after it.
 *                   Other shapes ignore the flag. Breaking the promise gives
 *                   stale values.
 *   key_length_late 0 (default): as above. Nonzero (with params_ready 0): the
 *                   caller says that the kernel launched immediately before
 *                   this call writes key_length, so an early read would be
 *                   stale; the compiled-shape kernel then takes no key_length
 *                   hint and prefetches each warp's window of new keys
 *                   instead, which skips the second pass a stale hint costs.
 *                   Results are the same either way.
 *
 * Limits: N, L >= 0; Di >= 1; 0 <= Dr <= Di, Dr even; Bcap >= 1; Bp >= 0.
 * Mean, normalisation and rotation in float32, one rounding to `in_dtype`.
 */
typedef struct kvr_qsa_args {
    const void* raw_index_keys;
    kvr_dtype in_dtype;
    int64_t N, L, Di;
    void* block_keys;
    int64_t Bcap;
    const int64_t* key_length;
    int64_t key_length_len;
    const void* rope_cos;
    const void* rope_sin;
    int64_t Dr;
    const void* k_norm_weight;
    const void* past_incomplete_raw_keys;
    const void* past_incomplete_rope;
    int64_t key_block_size;
    float eps;
    void* next_incomplete_raw_keys;
    void* next_incomplete_rope;
    int32_t* dev_status;
    kvr_qsa_rope rope_layout;
    const void* past_block_index_keys;
    int64_t Bp;
    int32_t params_ready;
    int32_t key_length_late;
} kvr_qsa_args;

kvr_status qsa_prepare(const kvr_qsa_args* args, cudaStream_t stream);

/*
 * Arguments of dynamic_quant(): DynamicQuant of q^N from "aclnnMlaPrologV3WeightNz"
 * ("Formula": dequantScaleQNope = RowMax(abs(q^N)) / 127,
 * q^N = round(q^N / dequantScaleQNope); "Shape restrictions": one scale per
 * (token, head), shape (T, N, 1)).
 *
 *   q_nope          [rows, Hckv] input, `in_dtype` (bf16 or f16); rows = T*N
 *                   (tokens x heads). Row r starts q_row_stride elements after
 *                   row r-1 (0 means Hckv).
 *   q_out           [rows, Hckv] int8 codes, dense.
 *   dequant_scale   [rows] float32 scales.
 *
 *   exact           0 (default) or 1, see below.
 *
 * Per row: dequant_scale = RowMax(|q|) / 127, rounded once to float32 (the
 * IEEE division), and code = round-half-even(q / (RowMax/127)) =
 * round-half-even(q * 127 / RowMax), clamped to [-127, 127]; an all-zero row
 * gets scale 0 and codes 0. With exact = 0 each code is computed from a
 * float32 reciprocal product and is within one code of that value (equal to
 * it unless q * 127 / RowMax lies within 2^-15 of a half-integer). With
 * exact = 1 those near-tie codes are recomputed from the exact rational, so
 * every code equals it; this costs about a third more time on bf16 rows,
 * where such quotients are common. Inputs are finite. Limits: rows >= 0,
 * Hckv >= 1; the outputs must not overlap the input (KVR_ERR_ALIAS).
 */
typedef struct kvr_dq_args {
    const void* q_nope;
    kvr_dtype in_dtype;
    int64_t rows, Hckv;
    int64_t q_row_stride;
    int8_t* q_out;
    float* dequant_scale;
    int32_t exact;
} kvr_dq_args;

kvr_status dynamic_quant(const kvr_dq_args* args, cudaStream_t stream);

/*
 * Arguments of query_rope(): the RoPE of q^R ("aclnnMlaPrologV3WeightNz",
 * "Formula", query path) by the interleaved formula of
 * "aclnnKvRmsNormRopeCache" ("Formulas (1) interleaveRope"), with positions of
 * several axes, as multimodal prompts have them.
 *
 *   q            [T, H, D] input, element type `dtype` (bf16 or f16), the last
 *                axis dense; row (t, h) starts at t * q_token_stride +
 *                h * q_head_stride elements.
 *   positions    int64 [axes, T], any sign and size.
 *   sections     HOST array of `axes` nonnegative counts that add up to D/2:
 *                the first sections[0] pairs turn by the position on axis 0,
 *                the next sections[1] by that on axis 1, and so on.
 *   base         pair i turns by position * base^(-2i/D); 1 <= base < 2^63.
 *   half_pairs   0: pair i is (x[2i], x[2i+1]); 1: (x[i], x[i + D/2]). Either way its
 *                results go to lanes i and i + D/2, as in kvr_qsa_rope.
 *   out          [T, H, D] `dtype`, strides as for q. Must not overlap q.
 *   cos_out, sin_out  optional out [T, D] `dtype`, dense (both or neither): the
 *                full-width tables of these positions, lanes i and i + D/2 equal,
 *                as kv_rmsnorm_rope_cache takes them.
 *
 * The angle's whole turns are dropped in 64-bit fixed point (base^(-2i/D) /
 * 2 pi is good to a multiple of 2^-50, so that an angle is off by at most
 * |position| * 2^-50 turns); cos and sin of the rest are float32, each
 * output is rounded once. Limits: T, H >= 0; D even, 2 <= D <= 256;
 * 1 <= axes <= 8; T * H * D < 2^40.
 */
#define KVR_MAX_AXES 8
typedef struct kvr_rope_args {
    const void* q;
    kvr_dtype dtype;
    int64_t T, H, D;
    int64_t q_token_stride, q_head_stride;
    const int64_t* positions;
    int64_t axes;
    const int64_t* sections;
    double base;
    int32_t half_pairs;
    void* out;
    int64_t out_token_stride, out_head_stride;
    void* cos_out;
    void* sin_out;
} kvr_rope_args;

kvr_status query_rope(const kvr_rope_args* args, cudaStream_t stream);

/*
 * Arguments of kv_cache_read(): for each token of an index, the two cache rows
 * that kv_rmsnorm_rope_cache() writes for it, side by side in one dense row.
 *
 *   ckv_cache, k_cache, their types, scales and dims, mode, index: as in
 *                kvr_kv_args. An 8-bit code is read as code / scale[c].
 *                An index entry may occur several times.
 *   out          [B, S, >= Dv + Dk] of `out_dtype` (bf16 or f16; a 16-bit cache
 *                has this type too); row t starts out_row_stride elements after
 *                row t - 1 (0 means Dv + Dk). The row of an entry -1 is left as
 *                it was; so is that of an entry out of range, which raises
 *                KVR_DEVERR_INDEX. Must not overlap an input.
 *
 * Decoded in float32 (the code times the correctly rounded 1/scale), rounded
 * once to out_dtype. Limits as kvr_kv_args, but Dk >= 0 (0: no k part; k_cache
 * may then be NULL) and odd widths are fine.
 */
typedef struct kvr_read_args {
    const void* ckv_cache;
    kvr_dtype ckv_dtype;
    const float* ckv_scale;
    int64_t ckv_scale_len;
    const void* k_cache;
    kvr_dtype k_dtype;
    const float* k_scale;
    int64_t k_scale_len;
    kvr_cache_mode mode;
    int64_t cache_d0, cache_d1;
    const int64_t* index;
    int64_t B, S, Dv, Dk;
    void* out;
    kvr_dtype out_dtype;
    int64_t out_row_stride;
    int32_t* dev_status;
} kvr_read_args;

kvr_status kv_cache_read(const kvr_read_args* args, cudaStream_t stream);

/*
 * Arguments of mla_attention(): for token j of sequence n and head h
 *
 *   s[i] = softmax_scale * (q_nope . c[i] + q_rope . k[i])      over the keys i it sees
 *   out  = sum_i softmax(s)[i] c[i]
 *
 * with c[i], k[i] the rows of key i of the sequence in ckv_cache and k_cache
 * (the absorbed form of latent attention: one key row for all heads, its
 * latent part is the value too).
 *
 *   q_nope, q_rope  [T, H, Dv] and [T, H, Dk], element type `dtype` (bf16 or
 *                f16), last axis dense, row (t, h) at t * token_stride +
 *                h * head_stride elements.
 *   query_start  int64 [N + 1]: the new tokens of sequence n are rows
 *                [query_start[n], query_start[n + 1]) of q and out. Rows outside
 *                every sequence are left as they were. A sequence where it
 *                decreases or leaves [0, T] is left out (KVR_DEVERR_QUERY); rows
 *                that two of the others then share get elements of either result.
 *   key_length   int64 [N]: keys of the sequence, its new tokens among them (as
 *                qsa_prepare's). A negative one, or one beyond the block table (the
 *                cache batch in Norm mode): the sequence is left out
 *                (KVR_DEVERR_KEY_LENGTH).
 *   causal       nonzero: with L new tokens and K keys, token j sees keys
 *                [0, K - L + j + 1), and nothing where that is empty (L > K).
 *                0: every token sees all K keys.
 *                Keys at or behind K are never used, whatever they hold. Those
 *                before K are taken to be finite: a NaN or an infinity in one may
 *                reach every token of its sequence, also one that does not see it
 *                (its weight there is zero, and zero times it is NaN).
 *   mode         KVR_CACHE_NORM: sequence n reads cache batch n (needs
 *                cache_d0 >= N; no block table). KVR_CACHE_PA_BSND or
 *                KVR_CACHE_PA_BLK_BSND: key i is in block
 *                block_table[n, i / d1] at i % d1.
 *   block_table  int64 [N, max_blocks]. An entry -1 leaves that block's keys out
 *                (nothing of them is read); so does one out of range, which
 *                raises KVR_DEVERR_INDEX if a token sees the block. Entries
 *                behind the last key are not used.
 *   ckv_dtype, k_dtype, ckv_scale, k_scale  as in kvr_kv_args; an 8-bit code
 *                stands for code / scale[c].
 *   out          [T, H, Dv] `dtype`, strides as for q. A token that sees no key
 *                gets zeros, and so does one whose every score is -inf. A query
 *                row that holds a NaN gives NaN in its output row and lse, and
 *                in no other.
 *   lse          optional out float32 [T, H]: log(sum_i exp(s[i])), -inf for a
 *                token that sees no key.
 *   workspace    device memory of kvr_mla_attention_workspace(args) bytes,
 *                32-byte aligned; it holds nothing between calls. Calls that can
 *                run at the same time need one each.
 *   dev_status   optional int32 device word (the bits above and
 *                KVR_DEVERR_TIMEOUT).
 *
 * Limits: T, H >= 0; 0 <= N < 2^31 - 512; T * H < 2^31; 1 <= Dv <= 1024; 1 <= Dk <= 256;
 * keys of a sequence <= 2^24 (one that has more is left out, KVR_DEVERR_KEY_LENGTH). Rows of
 * at most 512 + 64 channels, both multiples of 8 (of 16 in an 8-bit cache), on
 * 16-byte boundaries (q, out, caches; strides multiples of 8) and with H <= 65536
 * run on the tensor cores, all others on a plain kernel that is much slower. On the
 * tensor cores T * H / 128 * N * H * (keys + 1024) < 2^62, with the keys that the
 * block table (the cache batch in Norm mode) has room for.
 * Scores, softmax and sums are float32. The tensor-core kernel rounds each
 * probability for the second product, to `dtype`, or to float16 with an 8-bit
 * latent cache, whose products run on float16 (every code is exact there); a
 * float16 weight also loses up to 2^-32 of its row's largest weight. A
 * scale per channel goes into the query: q / scale[c] is rounded once, to
 * float16 for the latent part and to `dtype` for the rotary part, which moves a
 * score by up to one unit in the last place of that type (relative to the
 * terms' size) and lse with it; one scale for all channels rounds nothing more.
 * The output's sum on the tensor cores takes 16 keys an addition and cuts it off:
 * up to keys * 2^-27 of the terms' size where one CTA pair goes over all keys
 * (measured: 2^-10 of the output at 2^20 keys).
 * out, lse and workspace must not overlap an input or one another. The result
 * of a call does not change from run to run on one GPU.
 */
typedef struct kvr_mla_args {
    const void* q_nope;
    const void* q_rope;
    kvr_dtype dtype;
    int64_t T, H, Dv, Dk;
    int64_t q_nope_token_stride, q_nope_head_stride;
    int64_t q_rope_token_stride, q_rope_head_stride;
    int64_t N;
    const int64_t* query_start;
    const int64_t* key_length;
    kvr_cache_mode mode;
    int64_t cache_d0, cache_d1;
    const int64_t* block_table;
    int64_t max_blocks;
    const void* ckv_cache;
    kvr_dtype ckv_dtype;
    const float* ckv_scale;
    int64_t ckv_scale_len;
    const void* k_cache;
    kvr_dtype k_dtype;
    const float* k_scale;
    int64_t k_scale_len;
    float softmax_scale;
    int32_t causal;
    void* out;
    int64_t out_token_stride, out_head_stride;
    float* lse;
    void* workspace;
    int64_t workspace_bytes;
    int32_t* dev_status;
} kvr_mla_args;

kvr_status mla_attention(const kvr_mla_args* args, cudaStream_t stream);

/* Bytes of workspace that mla_attention(args) needs on the current device (0
 * where it needs none, or where args are not valid). Depends on T, H, the
 * widths, types, scale lengths, strides and alignments in *args, not on what
 * the device arrays hold; `workspace` itself is not looked at. */
int64_t kvr_mla_attention_workspace(const kvr_mla_args* args);

/*
 * Arguments of draft_tree(): the tokens that a draft proposes for a sequence form
 * a tree (or several) that continues its context.
 *
 *   query_start  int64 [N + 1]: the drafted tokens of sequence n are rows
 *                [query_start[n], query_start[n + 1]), as in mla_attention.
 *   parent       int64 [T]: the place, in its sequence, of the token that this one
 *                continues, before its own; -1: it continues the context. Any
 *                other entry counts as -1 and raises KVR_DEVERR_INDEX.
 *   tree_mask    out int64 [T, mask_words]: bit b % 64 of word b / 64 is set where
 *                token b of the sequence is the token itself or an ancestor.
 *   positions    optional out int64 [T]: position_start[n] + the number of
 *                ancestors, as query_rope and the prologue's tables take it.
 *   position_start  int64 [N], needed with positions.
 *   dev_status   optional int32 device word.
 *
 * A sequence where query_start decreases or leaves [0, T], or with more than
 * 64 mask_words tokens, is left out (KVR_DEVERR_QUERY). Rows of such a sequence
 * and rows outside every sequence are left as they were; rows that two of the
 * others then share get words of either. Limits: T >= 0,
 * 0 <= N < 2^31, 1 <= mask_words <= 64. The outputs must not overlap an input or
 * one another.
 */
typedef struct kvr_tree_args {
    int64_t T, N;
    const int64_t* query_start;
    const int64_t* parent;
    const int64_t* position_start;
    int64_t* tree_mask;
    int64_t mask_words;
    int64_t* positions;
    int32_t* dev_status;
} kvr_tree_args;

kvr_status draft_tree(const kvr_tree_args* args, cudaStream_t stream);

/*
 * Arguments of mla_tree_attention(): mla_attention() where token j of a sequence
 * with L new tokens and K keys sees the keys [0, K - L) and, for each bit b < L of
 * its words, key K - L + b (where that is not negative). Its own bit counts like
 * any other.
 *
 *   attention    as for mla_attention; `causal` is not looked at.
 *   tree_mask    int64 [T, mask_words], rows as those of q; must not overlap an
 *                output. A sequence with more than 64 mask_words tokens is left
 *                out (KVR_DEVERR_QUERY).
 *
 * Limits and workspace are those of mla_attention; mask_words >= 1.
 */
typedef struct kvr_mla_tree_args {
    kvr_mla_args attention;
    const int64_t* tree_mask;
    int64_t mask_words;
} kvr_mla_tree_args;

kvr_status mla_tree_attention(const kvr_mla_tree_args* args, cudaStream_t stream);

/*
 * Arguments of mla_key_weight(): the attention weight that each key of a sequence
 * receives from the sequence's tokens t and heads h,
 *
 *   weight[n, i] = decay * past[n, i] + sum_{t, h} exp(s[t, h, i] - lse[t, h])
 *
 * over the tokens that see key i, s as in mla_attention.
 *
 *   step         as for mla_attention, but `out` is not used and `lse` is read
 *                (float32 [T, H], needed): what mla_attention wrote for these queries,
 *                or any other logarithms. A row of -inf adds nothing, whatever
 *                its query holds (padding).
 *   weight       out float32: key i of sequence n at n * weight_stride + i, room
 *                for weight_len keys a sequence. Entries behind a sequence's last
 *                key, and those of sequences without tokens, are left as they were.
 *                A sequence with more than weight_len keys is left out
 *                (KVR_DEVERR_KEY_LENGTH). Keys of blocks that the table leaves
 *                out receive nothing: they get decay * past.
 *   past         float32, laid out with past_stride, read for the same keys: `weight`
 *                itself (with the same stride) to add up in place, another array that
 *                does not overlap it, or NULL: nothing is read.
 *   decay        factor of past.
 *
 * Limits are those of mla_attention, weight_len >= 0, strides >= weight_len;
 * `weight` must not overlap an input, the workspace or dev_status. Rows of at
 * most 512 + 64 channels, both multiples of 8 (of 16 in an 8-bit cache), on
 * 16-byte boundaries (q and the caches; strides multiples of 8) and with H <=
 * 65536 run on the tensor cores, all others on a plain kernel that is much
 * slower; the limits are there T * H <= 2^31 - 512 and, on work, (T * H / 32 + 2) *
 * (keys / 256 + 2) * N < 2^62. Scores and sums are float32. A query for a cache with scales per
 * channel is divided by them and held in 22 bits there; with one scale for all
 * latent channels the rotary part is multiplied by it and held in 16 bits (of
 * bf16) or 22. Keys within key_length need not be
 * finite: one that is not changes no weight but its own. The result of a call
 * does not change from run to run on one GPU.
 */
typedef struct kvr_key_weight_args {
    kvr_mla_args step;
    float* weight;
    int64_t weight_stride, weight_len;
    const float* past;
    int64_t past_stride;
    float decay;
} kvr_key_weight_args;

kvr_status mla_key_weight(const kvr_key_weight_args* args, cudaStream_t stream);

/* Bytes of workspace that mla_key_weight(args) needs on the current device (0
 * where it needs none, or where args are not valid), as
 * kvr_mla_attention_workspace. */
int64_t kvr_mla_key_weight_workspace(const kvr_key_weight_args* args);

/*
 * Arguments of kv_cache_select(): of the key_length[n] keys of a sequence, the
 * `keep` to keep. All, where they are no more than that; else the first `sink`,
 * the last `recent` and, of those between, the ones of largest weight: of equal
 * weights (-0 equals 0) the earlier, NaN above every number.
 *
 *   weight       float32: key i of sequence n at n * weight_stride + i, room for
 *                weight_len keys a sequence.
 *   key_length   int64 [N]. A negative one or one beyond weight_len: the sequence
 *                is left out (KVR_DEVERR_KEY_LENGTH), as if it had no keys.
 *   kept         out int64 [N, keep]: positions of the kept keys, ascending, then -1.
 *   kept_length  out int64 [N]: how many they are.
 *   kept_weight  optional out float32, row n at n * kept_weight_stride: the kept
 *                keys' weights in that order, then zeros up to kept_weight_len
 *                (>= keep).
 *   dev_status   optional int32 device word.
 *
 * Limits: 0 <= N < 2^27, weight_len <= 2^30, keep >= 1, sink, recent >= 0,
 * sink + recent <= keep < 2^31. The outputs must not overlap an input or one
 * another.
 */
typedef struct kvr_select_args {
    const float* weight;
    int64_t weight_stride, weight_len;
    int64_t N;
    const int64_t* key_length;
    int64_t keep, sink, recent;
    int64_t* kept;
    int64_t* kept_length;
    float* kept_weight;
    int64_t kept_weight_stride, kept_weight_len;
    int32_t* dev_status;
} kvr_select_args;

kvr_status kv_cache_select(const kvr_select_args* args, cudaStream_t stream);

/*
 * Arguments of kv_cache_compact(): rows of a sequence moved together in place, in
 * both caches: key start[n] + i becomes what key kept[n, i] was, for
 * i < kept_length[n].
 *
 *   ckv_cache, k_cache, ckv_dtype, k_dtype, mode, cache_d0, cache_d1,
 *   block_table, max_blocks  the caches as in mla_attention, any two types; rows
 *                move as they are, so scales are not needed. Dk >= 0 (0: no k part;
 *                k_cache may then be NULL).
 *   kept         int64 [N, kept_len], ascending in each row, kept[n, i] >=
 *                start[n] + i, as kv_cache_select gives it (start 0) or as the
 *                places of an accepted branch of a drafted tree (start: the keys
 *                before the tree). An entry that is not, or that lies behind the block
 *                table's keys, and a row whose block the table does not name:
 *                that row is not written (KVR_DEVERR_INDEX), and where the order is
 *                broken the sequence's other rows get an unspecified mix of rows.
 *                A row with kept[n, i] = start[n] + i is not touched.
 *   kept_length  int64 [N], at most kept_len.
 *   start        int64 [N], or NULL for 0. A negative start or kept_length, or one
 *                too large: the sequence is left out (KVR_DEVERR_KEY_LENGTH).
 *   dev_status   optional int32 device word.
 *
 * A row that moves must be of one sequence alone: blocks that sequences share have
 * to lie within keys that stay. Limits: 0 <= N < 2^31, Dv >= 1, kept_len >= 0,
 * block-table keys < 2^31. kept, kept_length, start and the table must not overlap
 * the caches, nor the caches one another.
 */
typedef struct kvr_compact_args {
    void* ckv_cache;
    kvr_dtype ckv_dtype;
    void* k_cache;
    kvr_dtype k_dtype;
    kvr_cache_mode mode;
    int64_t cache_d0, cache_d1;
    const int64_t* block_table;
    int64_t max_blocks;
    int64_t N, Dv, Dk;
    const int64_t* kept;
    int64_t kept_len;
    const int64_t* kept_length;
    const int64_t* start;
    int32_t* dev_status;
} kvr_compact_args;

kvr_status kv_cache_compact(const kvr_compact_args* args, cudaStream_t stream);

/* Measurement helper (no counterpart on the pages): a 16-byte vectorised
 * device-to-device copy of `bytes` bytes (a multiple of 16, both pointers
 * 16-byte aligned), used to measure the achievable HBM bandwidth in the same
 * process as the kernels above. */
kvr_status kvr_device_copy(void* dst, const void* src, int64_t bytes, cudaStream_t stream);

/* Failure-detection check (no counterpart on the pages): one small kernel
 * waits, the way the pipeline kernels wait on their copies, for an mbarrier
 * phase that never completes (it expects bytes that no copy delivers). It
 * gives up after `limit_ns` nanoseconds (1e3 .. 1e9), or after
 * `abort_after_ns` (0 = never; at most limit_ns) when a second warp raises
 * the abort flag the pipelines use, then ORs KVR_DEVERR_TIMEOUT into the
 * device word *dev_status and returns: nothing traps and the context stays
 * usable. Asynchronous on `stream`. */
kvr_status kvr_check_bounded_wait(int32_t* dev_status, int64_t limit_ns, int64_t abort_after_ns, cudaStream_t stream);

/* Test helper (no counterpart on the pages): a late producer of device
 * words. One small kernel, launched with programmatic dependent launch like
 * the calls above, waits for its own predecessor on `stream`, lets the next
 * launch on `stream` start at once, spins for `delay_ns` nanoseconds
 * (0 .. 1e8) and only then copies `count` (0 .. 2^20) int64 words from the
 * device array `src` to the device array `dst` (both 8-byte aligned, not
 * overlapping; the caller keeps both alive until the stream has passed the
 * kernel). A call launched right after it therefore starts while `dst` still
 * holds its old values, and must see the new ones after its dependency wait:
 * the check that qsa_prepare's default form takes key_length only after the
 * wait (its earlier read is a prefetch hint). Returns KVR_ERR_SHAPE for a
 * count or delay out of range or a misaligned pointer, KVR_ERR_NULL for a
 * null pointer (count > 0), KVR_ERR_ALIAS for overlapping arrays; count 0
 * launches nothing. Asynchronous on `stream`. */
kvr_status kvr_store_after_delay(int64_t* dst, const int64_t* src, int64_t count, int64_t delay_ns,
                                 cudaStream_t stream);

/* Debug validation of kv_rmsnorm_rope_cache's index (off by default; the
 * environment variable KVR_DEBUG_VALIDATE=1 turns it on at the first call,
 * this call sets it either way, for every thread). When on, each
 * kv_rmsnorm_rope_cache / kv_rmsnorm_rope_cache_staged call copies its index
 * to the host, synchronising `stream`, and returns KVR_ERR_INDEX without
 * launching when an entry is out of range or two tokens name the same cache
 * row ("aclnnKvRmsNormRopeCache", "Restrictions on index": distinct within a
 * batch in Norm mode, anywhere in the paged modes; in PA_BLK_BSND every
 * token's row is checked and must stay inside its entry's block). Without
 * it, repeated rows leave an unspecified winner and out-of-range entries are
 * skipped and reported through dev_status. A call made while its stream is
 * being captured into a CUDA graph is not checked. For debugging only: the
 * copy and the synchronisation cost far more than the call. */
void kvr_set_debug_validate(int on);

/* Static description of a status code (never NULL). */
const char* kvr_status_string(kvr_status status);

/* KVR_ABI_VERSION of the loaded library. */
int kvr_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KVR_H */
