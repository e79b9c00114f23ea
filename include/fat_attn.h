/*
 * fat_attn.h -- C ABI of the GB300 (sm_103a) fused attention forward pass with
 * the tensorized online softmax.
 *
 * Operation (every entry point): for each batch b, head h and query row i,
 *
 *     O[b,h,i,:] = sum_j softmax_j(scale * Q[b,h,i,:] . K[b,h,j,:]) V[b,h,j,:]
 *     LSE[b,h,i] = ln sum_j exp(scale * Q[b,h,i,:] . K[b,h,j,:])
 *
 * over keys j = 0..N-1, or j = 0..i with the causal mask.  This is the fused
 * attention flow of "FlashAttention-T: Towards Fully Tensorized Attention by
 * Exploiting Tensor-Vector Parallelism" (papercache.org summary, section A3,
 * Fig. 2: one output row block per worker, S and P kept on chip), with the
 * tensorized online softmax of its section A2 (surrogate maximum over X-row
 * tiles, the equation defining m_hat; Algorithm 1 steps 1-7).
 *
 * Conventions shared by all entry points
 *  - Pointers are DEVICE pointers owned by the caller; the library never
 *    allocates, frees or keeps them.  Tensors are contiguous row-major:
 *    q, k, v [B, H, N, d] (bf16, or e4m3 for the fp8 entry point); o fp32
 *    [B, H, N, d]; lse fp32 [B, H, N] (natural log, in units of the scaled
 *    logits).  q, k, v, o and lse must be 16-byte aligned.
 *  - d is 64 or 128; X (rows sharing one surrogate maximum) is 16, 32, 64 or
 *    128; B, H, N >= 1 (any N: a ragged last tile is masked).
 *  - Arguments are validated before anything is launched; on failure nothing
 *    runs and a negative fat_status is returned.
 *  - The work is enqueued asynchronously on `stream` (0 = legacy default
 *    stream).  The library never synchronises, except in
 *    fat_check_device_error().
 *  - Device-side waits are bounded.  A wait that runs out stops the kernel,
 *    leaves o/lse unspecified and records FAT_ERR_DEVICE_TIMEOUT in a device
 *    error word that fat_check_device_error() reports.
 *  - Calls are re-entrant; the only library state is a per-device cache of
 *    the driver's tensor-map encoder and kernel attributes.
 */
#ifndef FAT_ATTN_H_
#define FAT_ATTN_H_

#include <stddef.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FAT_OK = 0,
  FAT_ERR_INVALID_ARG = -1,    /* null pointer, bad size, bad d / X, bad scale */
  FAT_ERR_UNSUPPORTED = -2,    /* a valid request this build does not implement */
  FAT_ERR_ALIGNMENT = -3,      /* a tensor is not 16-byte aligned */
  FAT_ERR_LAUNCH = -4,         /* CUDA reported an error while setting up or launching */
  FAT_ERR_DEVICE_TIMEOUT = -5, /* a bounded device wait ran out (see fat_check_device_error) */
  FAT_ERR_ARCH = -6,           /* the current device is not sm_103 */
  FAT_ERR_INDEX = -7           /* a kernel met a page, slot or length outside the cache or the
                                  page table (see fat_check_device_error) */
} fat_status;

typedef enum { FAT_VARIANT_TENSOR = 0, FAT_VARIANT_VEC = 1 } fat_variant;
/* Input type of q, k, v (fat_attn_fwd_ex): bf16; e4m3 with per-tensor
 * descales (d = 128 only); fp16 (the FA-T summary's FP16-FP32 setting, A4).
 * P~ takes the input type for the O += P~ V MMA (fp16 P~ as 2^(Z+15), e4m3 as
 * 2^(Z+8), to use those formats' ranges; the factor is taken off LSE). */
typedef enum { FAT_DTYPE_BF16 = 0, FAT_DTYPE_E4M3 = 1, FAT_DTYPE_FP16 = 2 } fat_dtype;

/*
 * Where the row sum l of Algorithm 1 step 7 is formed in the tensorized
 * variant.  FAT_LMODE_VECTOR (default): fp32 sum of the unrounded P~ on the
 * vector units (packed f32x2 adds).  FAT_LMODE_TENSOR: on the tensor pipe as
 * the bf16-rounded P~ times a block of ones, plus a per-tile correction of
 * the dominant term's rounding; O stays consistent with l, but LSE can then
 * be off by up to ~2^-9 when a few comparable terms dominate a row.
 */
typedef enum { FAT_LMODE_VECTOR = 0, FAT_LMODE_TENSOR = 1 } fat_lmode;

/*
 * Where the subtraction of Algorithm 1 steps 4-5 (Z = log2(e) * scale * S -
 * m_hat) happens in the tensorized variant.  FAT_ZMODE_VECTOR (default): one
 * packed FMA per pair of scores on the vector units.  FAT_ZMODE_TENSOR (the
 * tensor-pipe half of the "AllTensor" variant of the page's ablation, Fig. 10):
 * S = Q K^T gets one more 16-deep K step, a bias tile against a tile of ones,
 * so the MMA itself writes S + b with b = -m_ref / (log2(e) * scale) rounded
 * to bf16, m_ref being the surrogate maximum settled three K/V tiles earlier
 * (the latest one known when that S is queued).  The multiply by
 * log2(e) * scale and the remaining offset log2(e) * scale * b + m_hat stay
 * one packed FMA per pair, so no vector instruction is saved, and the MMA does 1/8 (d = 128)
 * or 1/4 (d = 64) more work on S.  Requires the tensorized variant, X = 128
 * and bf16 inputs; anything else returns FAT_ERR_UNSUPPORTED.
 */
typedef enum { FAT_ZMODE_VECTOR = 0, FAT_ZMODE_TENSOR = 1 } fat_zmode;

/*
 * How query tiles (128 rows of one (b, h): the row blocks of the page's
 * section A3, one per worker) map to thread blocks.  FAT_BLOCKS_AUTO
 * (default): one thread block per SM takes tiles in turn, so the next tile's
 * Q and first K tiles load, and its first S tiles run on the tensor pipe,
 * while the last tile's output is normalised and stored; split-KV calls use
 * one block per tile.  FAT_BLOCKS_PER_TILE: one thread block per tile, in the
 * same order (for comparison).  The results are the same either way.
 */
typedef enum { FAT_BLOCKS_AUTO = 0, FAT_BLOCKS_PER_TILE = 1 } fat_block_mode;

/*
 * Tensorized online softmax (section A2 of the page above).
 *   - m_hat: per X-row tile, the maximum of the row maxima seen so far
 *     (Algorithm 1 step 1), kept as an integer number of binades so that the
 *     rescale factor exp(m_hat_old - m_hat) of steps 2-3 is an exact power of
 *     two shared by the tile;
 *   - Z = log2(e) * scale * S - m_hat, P~ = exp2(Z) (steps 4-6);
 *   - O is rescaled in tensor memory by the vector units, once per tile and
 *     only when m_hat grew (for X = 128 one factor for the whole tile);
 *   - the row sum l of step 7 is an fp32 sum on the vector units (see
 *     fat_lmode for the tensor-pipe alternative);
 *   - rows whose surrogate maximum exceeds their exact maximum by more than
 *     the underflow threshold (default 64 binades for bf16 P~, 29 for fp16,
 *     14 for e4m3),
 *     or whose sum is zero, are detected; their 128-row block is recomputed
 *     with one-row tiles (X = 1: each row's own maximum rounded up to a whole
 *     binade, so no row can underflow) -- the optional fallback of the
 *     all-underflow discussion -- after the thread block's other tiles,
 *     overwriting the block's O and LSE.
 * q, k, v: bf16.  Returns a fat_status.
 */
int fat_attn_fwd(const void* q, const void* k, const void* v, float* o, float* lse, int B, int H,
                 int N, int d, int causal, float scale, int X, cudaStream_t stream);

/*
 * Vector-softmax ablation baseline (the "FA2" arm of the page's Fig. 10
 * ablation): exact per-row maximum, per-row rescale of O whenever a row
 * maximum grows, row sum accumulated on the vector units.  Same pipeline,
 * tiling and signature as fat_attn_fwd; X is validated but unused.
 */
int fat_attn_fwd_vec(const void* q, const void* k, const void* v, float* o, float* lse, int B,
                     int H, int N, int d, int causal, float scale, int X, cudaStream_t stream);

/*
 * FP8 (e4m3) inputs with per-tensor fp32 descales (real value = code * descale),
 * fp32 accumulation, the tensorized softmax of fat_attn_fwd.  (The page
 * evaluates FP8-FP32 attention in its section A4.)  d must be 128.  P~ is
 * stored as e4m3 scaled by 2^8 (largest term <= 256 < 448; the factor cancels
 * in O / l and is removed from LSE); O is rescaled on the vector side.
 * Descales must be finite and > 0.
 */
int fat_attn_fwd_fp8(const void* q, const void* k, const void* v, float q_descale,
                     float k_descale, float v_descale, float* o, float* lse, int B, int H, int N,
                     int d, int causal, float scale, int X, cudaStream_t stream);

/*
 * Split-KV forward (decode and long-key shapes): Nq query rows against Nk
 * keys per (b, h); q [B, H, Nq, d], k and v [B, H, Nk, d] (bf16), o fp32
 * [B, H, Nq, d], lse fp32 [B, H, Nq].  Causal keeps key j for query i iff
 * j <= i + Nk - Nq (the queries are the last Nq positions; requires
 * Nk >= Nq).  The key range is cut into up to num_splits ranges of whole
 * 128-key tiles (1 <= num_splits <= 64), each computed by its own thread
 * blocks with the tensorized online softmax of fat_attn_fwd; their partial
 * O and LSE go to `workspace` (device memory owned by the caller, at least
 * fat_attn_splitkv_workspace_bytes(B, H, Nq, d, num_splits) bytes; may be
 * NULL when a single range results) and are merged by LSE weights:
 * LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.  The merge is
 * the exact identity behind the page's online softmax (per-block maxima
 * and sums combined afterwards, section A3 / Fig. 2).  Calls sharing a
 * workspace must not overlap on the device.
 */
int fat_attn_fwd_splitkv(const void* q, const void* k, const void* v, float* o, float* lse, int B,
                         int H, int Nq, int Nk, int d, int causal, float scale, int X,
                         int num_splits, void* workspace, size_t workspace_bytes,
                         cudaStream_t stream);

/* Workspace size for fat_attn_fwd_splitkv (0 for invalid arguments). */
size_t fat_attn_splitkv_workspace_bytes(int B, int H, int Nq, int d, int num_splits);

/* A split count giving about eight thread blocks per SM of the current device
 * (at least four 128-key tiles per split). */
int fat_attn_splitkv_default_splits(int B, int H, int Nq, int Nk);

/*
 * fat_attn_fwd_splitkv without any device allocation, for callers that
 * cannot allocate device memory at the time of the call (their process gives
 * all device memory to its own pool at start-up, or they must not call
 * cudaMalloc / cudaFree, which can block or synchronise the device).  The
 * pages have no counterpart: this is a convenience of this library.
 *
 * Same arguments and results as fat_attn_fwd_splitkv, minus the workspace:
 * the partial results use a fixed array of FAT_NOALLOC_SCRATCH_BYTES that
 * belongs to the library's device image, so every GPU that loads the library
 * holds that memory until the process exits.  Requests whose workspace
 * (fat_attn_splitkv_workspace_bytes) exceeds it return FAT_ERR_INVALID_ARG
 * and launch nothing.  The first call on a device looks up the array's
 * device address (cudaGetSymbolAddress); make that first call before any
 * stream capture.  If the lookup fails, that call returns FAT_ERR_LAUNCH and
 * the next call on the device tries again.  Nothing in the array needs to
 * start at zero (each call
 * writes every entry it reads), but all calls share it and it keeps the last
 * call's contents: calls whose work overlaps on the device race with each
 * other, so serialise them (for example on one stream).
 */
#define FAT_NOALLOC_SCRATCH_BYTES (16u << 20)
int fat_attn_fwd_splitkv_noalloc(const void* q, const void* k, const void* v, float* o,
                                 float* lse, int B, int H, int Nq, int Nk, int d, int causal,
                                 float scale, int X, int num_splits, cudaStream_t stream);

/*
 * fat_attn_fwd on host-resident tensors: q, k, v bf16 [B, H, N, d] and o, lse
 * fp32 ([B, H, N, d], [B, H, N]) in page-locked host memory.  The problem is
 * streamed through the device in chunks of heads_per_chunk heads (heads are
 * independent and contiguous): the copy to the device of one chunk, the
 * kernel of the previous one and the copy back of the one before overlap on
 * three internal streams, through three chunk slots in `workspace` (device
 * memory owned by the caller, at least fat_attn_fwd_host_workspace_bytes(...)
 * bytes).  Every copy is one cudaMemcpyAsync.  The work starts after what is
 * already queued on `stream`, and `stream` waits for the last copy back, so
 * the results are on the host once `stream` has completed.  heads_per_chunk
 * <= 0 picks about eight chunks.  Calls sharing a workspace, or running on
 * the same device from several host threads, must not overlap.  No
 * counterpart on the pages.
 */
int fat_attn_fwd_host(const void* q, const void* k, const void* v, float* o, float* lse, int B,
                      int H, int N, int d, int causal, float scale, int X, int heads_per_chunk,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace size for fat_attn_fwd_host (0 for invalid arguments). */
size_t fat_attn_fwd_host_workspace_bytes(int B, int H, int N, int d, int heads_per_chunk);

/* Every knob of the entry points above in one struct (tests and ablations). */
typedef struct fat_params {
  const void* q;
  const void* k;
  const void* v;
  float* o;
  float* lse;
  int B, H, N, d;
  int causal;
  float scale;
  int X;
  int variant;                        /* fat_variant */
  int dtype;                          /* fat_dtype */
  int l_mode;                         /* fat_lmode (tensorized variant only) */
  float q_descale, k_descale, v_descale; /* e4m3 only; ignored otherwise */
  float underflow_log2_threshold;     /* <= 0: default (64 binades for bf16 P~, 29 for fp16,
                                         14 for e4m3) */
  int* fallback_rows;                 /* nullable device int: += number of rows recomputed */
  unsigned long long wait_poll_limit; /* 0: no cap on polls of one device wait */
  unsigned long long wait_timeout_ns; /* 0: default of 4 s per device wait */
  cudaStream_t stream;
  /* nullable device buffer of FAT_TRACE_WORDS u64 (8-byte aligned): SM-clock
   * stamps of the first thread block's pipeline phases on its first query
   * tile, for measuring how long the tensor pipe waits for the softmax (see
   * the trace layout below) */
  unsigned long long* trace;
  int z_mode;                         /* fat_zmode (tensorized variant only) */
  int block_mode;                     /* fat_block_mode */
} fat_params;

/*
 * Trace layout (first thread block, first query tile, first pass): word
 * (e * 2 + t) * FAT_TRACE_ITERS + j holds the clock of event e at K/V tile j
 * (< FAT_TRACE_ITERS); t = the softmax set that takes tile j (j % 2) for the
 * softmax events, 0 for the MMA issuer's: e = 0 softmax received S_j; 1
 * softmax computed m_hat; 2 softmax published P_j; 3 MMA issuer saw P_j; 4
 * MMA issuer queued O += P_j V and S_{j+3}.  Word FAT_TRACE_WORDS-2: kernel
 * start; FAT_TRACE_WORDS-1: end of that tile's softmax epilogue.  Words of events
 * that did not happen are left untouched.
 */
#define FAT_TRACE_ITERS 128
#define FAT_TRACE_EVENTS 5
#define FAT_TRACE_WORDS (FAT_TRACE_EVENTS * 2 * FAT_TRACE_ITERS + 2)

int fat_attn_fwd_ex(const fat_params* p);

/*
 * Backward pass by recomputation (the v1 recap of the FA-T blog, "从融合到
 * 张量化：FlashAttention 演进脉络": only O and the softmax statistics are kept
 * from the forward pass).  For O = softmax(scale Q K^T [+ causal]) V and an
 * upstream gradient dout, writes the gradients of sum(O * dout):
 *   P = exp(scale S - LSE), D_i = sum_d dout_id O_id,
 *   dV = P^T dout, dS = P * (dout V^T - D), dQ = scale dS K, dK = scale dS^T Q.
 * q, k, v, dout: bf16 [B, H, N, d]; o, lse: the fp32 outputs of a forward
 * call on the same q, k, v (any variant: they are exact up to rounding);
 * dq, dk, dv: fp32 [B, H, N, d], overwritten (dq is cleared on `stream`
 * first and accumulated across key blocks with TMA reduce-adds in no fixed
 * order, so its low-order bits may differ from run to run).  d is 64 or 128.  P and dS enter their
 * MMAs as bf16, with fp32 accumulation.  workspace: device memory owned by
 * the caller, at least fat_attn_bwd_workspace_bytes(B, H, N) bytes (D and
 * log2(e) LSE per row); calls sharing it must not overlap on the device.
 * q, k, v, dout, o, dq, dk, dv must be 16-byte aligned, lse 4-byte aligned.
 * Returns a fat_status; nothing is launched when validation fails.
 */
int fat_attn_bwd(const void* q, const void* k, const void* v, const float* o, const float* lse,
                 const void* dout, float* dq, float* dk, float* dv, int B, int H, int N, int d,
                 int causal, float scale, void* workspace, size_t workspace_bytes,
                 cudaStream_t stream);

/* Workspace size for fat_attn_bwd (0 for invalid arguments). */
size_t fat_attn_bwd_workspace_bytes(int B, int H, int N);

/* ------------------------------------------------------------------------
 * Serving over a paged key-value cache
 * ------------------------------------------------------------------------
 * Keys and values of a pool of pages, [num_pages, heads, page_size, d], and a
 * page table that says which page holds positions [i * page_size,
 * (i + 1) * page_size) of which sequence.  Query heads come in groups:
 * q_heads is a multiple of heads, and query head h reads cached head
 * h / (q_heads / heads).
 *
 *  - page_size is a power of two, 16 to 1024; d is 64 or 128.
 *  - dtype: FAT_DTYPE_BF16, FAT_DTYPE_FP16, or FAT_DTYPE_E4M3 with one scale
 *    byte e per row (k_scale, v_scale: contiguous [num_pages, heads,
 *    page_size]): the row's values are code * 2^(e - 127), e = 1..254; e = 255
 *    marks a row that holds an inf or a NaN, and every element reads as NaN.
 *  - Strides are in elements, between pages, heads and tokens (the d elements
 *    of a row are adjacent); each is a multiple of 16 bytes below 4 GiB, and
 *    so are those of q and of the tokens (FAT_ERR_ALIGNMENT otherwise).  Any
 *    order of the three dimensions is allowed, as are k and v as parts of one
 *    tensor.
 *  - k and v are 16-byte aligned, the scales 16-byte aligned.
 *
 * Indexes that live on the device (pages, lengths, slots) cannot be checked
 * before the launch.  The kernels check them: a page outside [0, num_pages),
 * a length below 0 or above width * page_size, or a slot beyond the cache is
 * never used as an address; it sets FAT_ERR_INDEX for fat_check_device_error,
 * and that sequence's (or token's) results are unspecified.  Table entries
 * behind a sequence's last page are not used.
 *
 * A captured graph replays these calls with whatever the tensors hold then
 * (lengths, pages and slots included); make the first call of each kind, which
 * loads its kernels, before any stream capture.
 */
typedef struct fat_kv_cache {
  void* k;
  void* v;
  unsigned char* k_scale; /* e4m3 only, else ignored */
  unsigned char* v_scale;
  long long num_pages;
  int heads, page_size, d;
  int dtype; /* fat_dtype */
  long long k_page_stride, k_head_stride, k_token_stride;
  long long v_page_stride, v_head_stride, v_token_stride;
} fat_kv_cache;

typedef struct fat_page_table {
  const int* pages;    /* page of position i * page_size of sequence b: pages[b * stride + i] */
  long long stride;    /* >= width */
  int width;           /* entries of a sequence; width * page_size <= 2^30 */
  int batch;           /* sequences */
  const int* seq_lens; /* [batch] cached positions of each sequence (0 allowed) */
} fat_page_table;

/*
 * Store new tokens: k, v [tokens, heads, d] (bf16 or fp16, strides in
 * elements, rows 16-byte aligned) go to slots[t] = page * page_size + place
 * of the cache.  slots[t] < 0 skips the token (padding).  A cache of 16-bit
 * type takes its own type as it is.  An e4m3 cache takes either: a row's
 * scale is the least power of two that brings its largest magnitude to at
 * most 448 (1 for a row of zeros), so dividing by it is exact and each
 * element is rounded once, to nearest even.  The slots of one call must
 * differ.  tokens = 0 is allowed; tokens * heads is below 2^31 - 2^16.
 */
int fat_kv_write(const fat_kv_cache* cache, const void* k, const void* v, int dtype,
                 long long k_token_stride, long long k_head_stride, long long v_token_stride,
                 long long v_head_stride, const long long* slots, int tokens,
                 cudaStream_t stream);

/*
 * Read sequences back: k, v become contiguous [batch, heads, max_len, d]
 * tensors of `dtype` (bf16 or fp16; the cache's own type unless it is e4m3),
 * 16-byte aligned.  Rows from a sequence's length on are zeros; positions from
 * max_len (at most 2^30) on are left out.
 */
int fat_kv_read(const fat_kv_cache* cache, const fat_page_table* table, void* k, void* v,
                int dtype, int max_len, cudaStream_t stream);

/*
 * Attention of one new query token per sequence over its cached positions:
 *     z_j = scale * q[b,h] . K_j,  o[b,h] = sum_j softmax_j(z) V_j,
 *     lse[b,h] = ln sum_j exp(z_j),   j = 0 .. seq_lens[b] - 1.
 * q: [batch, q_heads, d] of `dtype` (bf16 or fp16, the cache's own type
 * unless it is e4m3), strides in elements, rows 16-byte aligned; o: contiguous
 * [batch, q_heads, d] of the same type, rounded once; lse: fp32 [batch,
 * q_heads].  A sequence of length 0 gives o = 0 and lse = -inf.
 * workspace: at least fat_attn_decode_workspace_bytes(...) bytes of device
 * memory, 16-byte aligned, any contents; calls sharing it must not overlap on
 * the device.  It may be NULL if width * page_size <= FAT_DECODE_DIRECT: no
 * sequence is split then.
 *
 * The weights of the values of an fp16 cache reach down to 2^-36 of a head's
 * largest, those of an e4m3 cache to 2^-36 of its largest product of weight and
 * row scale (rows of zeros left aside, whatever their scale byte): what is
 * below adds nothing, and each weight is off by no more than that besides its
 * own rounding.  With scales as fat_kv_write sets them that is far below an
 * output's rounding, unless a column is (nearly) zero in the rows that dominate.
 * An infinite value of an fp16 cache gives NaN where its weight is below 2^-34
 * of the largest.
 */
#define FAT_DECODE_DIRECT 512
int fat_attn_decode_paged(const fat_kv_cache* cache, const fat_page_table* table, const void* q,
                          int dtype, long long q_batch_stride, long long q_head_stride,
                          int q_heads, float scale, void* o, float* lse, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/* Workspace size for fat_attn_decode_paged (0 for invalid arguments). */
size_t fat_attn_decode_workspace_bytes(int batch, int q_heads, int kv_heads, int d);

/*
 * Bounds of the keys of each block (a block is one page): bounds [num_pages,
 * heads, 2, d], contiguous, 16-byte aligned, of `dtype` (the cache's own
 * type; bf16 or fp16 for an e4m3 cache), holds the elementwise minimum
 * (bounds[..., 0, :]) and maximum (bounds[..., 1, :]) of the block's keys.
 * This call renews the blocks that hold any of the last new_tokens positions
 * of each sequence (new_tokens >= 1; all blocks if it is at least the
 * length), over their positions below the length; other blocks keep what
 * they have.  A NaN key makes its bound NaN; a value of an e4m3 cache that
 * `dtype` cannot hold is rounded to nearest.  A page that stands in several
 * sequences' lines (a shared prefix) must be filled to the same position in
 * each of them whose newest positions touch it, as a page is copied before one
 * of its sequences goes on in it; else its bounds are unspecified, a mixture of
 * theirs.  cache->v is not used.
 */
int fat_kv_block_bounds(const fat_kv_cache* cache, const fat_page_table* table, int new_tokens,
                        void* bounds, int dtype, cudaStream_t stream);

/*
 * The score of every block of every sequence: scores[b, g, i], fp32
 * [batch, kv_heads, width], is the largest over the query heads h of group g of
 *     sum_c max(q[b,h,c], 0) hi_c + min(q[b,h,c], 0) lo_c,
 * an upper bound of q . k over the block's keys, with lo and hi the bounds of
 * the page at pages[b, i]; -inf behind the sequence's last block.  (Up to the
 * rounding of its fp32 sum; and where fp16 bounds of an e4m3 cache were rounded,
 * beyond fp16's range or among its subnormals, a key may lie outside them.  An
 * infinite bound times a zero of q+ or q- is NaN, which counts as the highest.)  q as in
 * fat_attn_decode_paged, of the bounds' type.
 */
int fat_kv_block_scores(const void* q, int dtype, long long q_batch_stride,
                        long long q_head_stride, int q_heads, const void* bounds,
                        long long num_pages, int kv_heads, int page_size, int d,
                        const fat_page_table* table, float* scores, cudaStream_t stream);

/*
 * Attention of one new query token per sequence over chosen blocks: for each
 * (sequence, cached head) the num_blocks blocks with the highest scores
 * (fp32 [batch, kv_heads, width], from fat_kv_block_scores or any other
 * source), or all if the sequence has no more.  The last last_blocks blocks
 * (the newest tokens) and then the first first_blocks ones are taken ahead of
 * all others; NaN counts as the highest score, and of equal ones the lower
 * index is taken.  blocks: int32 [batch, kv_heads, num_blocks], receives the
 * chosen block indexes in rising order, then -1.  Everything else as in
 * fat_attn_decode_paged; workspace: fat_attn_decode_sparse_workspace_bytes.
 */
int fat_attn_decode_sparse(const fat_kv_cache* cache, const fat_page_table* table, const void* q,
                           int dtype, long long q_batch_stride, long long q_head_stride,
                           int q_heads, const float* scores, int num_blocks, int first_blocks,
                           int last_blocks, float scale, void* o, float* lse, int* blocks,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace size for fat_attn_decode_sparse (0 for invalid arguments). */
size_t fat_attn_decode_sparse_workspace_bytes(int batch, int q_heads, int kv_heads, int d,
                                              int num_blocks);

/* Human-readable name of a fat_status value (static string). */
const char* fat_status_string(int status);

/*
 * Synchronises `stream`, then reads and clears the device error word of the
 * current device.  Returns FAT_ERR_DEVICE_TIMEOUT if a kernel of this library
 * stopped on a bounded wait since the last check, else FAT_ERR_INDEX if one
 * met an index outside its tensor, FAT_ERR_LAUNCH if the synchronisation
 * itself failed, FAT_OK otherwise.
 */
int fat_check_device_error(cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FAT_ATTN_H_ */
