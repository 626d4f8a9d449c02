/*
 * libmsa -- the MiniMax Sparse Attention (MSA) hot path on one NVIDIA GB300
 * (sm_103a), as a C ABI.
 *
 * The method (sources named by page title and section):
 *   [README] "MiniMax-AI/MSA" README (pigsec.cn mirror), section "Usage":
 *            a dense proxy pass (plan with num_kv_heads=1,
 *            output_maxscore=True) gives a per-block max score;
 *            sparse_topk_select(max_score, topk, num_valid_pages) turns it
 *            into kv_block_indexes; a plan with kv_block_num=topk runs
 *            attention over only those blocks of the paged K/V
 *            (k_pages, v_pages, kv_indices), page_size 128.
 *   [STACKS] same README, section "Stacks": paged FP8 decode
 *            (SparseDecodePagedAttentionWrapper) next to BF16 sparse prefill.
 *   [FLASH]  iitog.ru, "Flash-MSA: open kernels for training models with
 *            sparse attention on millions of tokens": whole 128-token blocks
 *            chosen by max-pooling proxy scores; GQA main attention; one
 *            block set per proxy head / GQA group; the token's own block is
 *            always visible; indexes cached from the forward feed the
 *            backward; the KL-loss gradient with respect to a proxy score is
 *            p_proxy - p_main.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every tensor argument is a DEVICE pointer to a dense row-major array
 *    owned by the caller; layouts are given per call.  The library never
 *    frees or retains them past the call.
 *  - Compute calls enqueue work on `stream` and return without waiting; they
 *    allocate nothing (any scratch lives in the plan, allocated once by
 *    msa_plan) and never synchronise the host.
 *  - Tiles: a sequence with qo_len query rows and kv_len keys (qo_len <=
 *    kv_len) places row r at key position kv_len - qo_len + r (bottom-right
 *    causal alignment) and row r sees key k iff k <= that position.  Query
 *    rows are cut into tiles of 128 rows per sequence; tiles are numbered
 *    across the batch in sequence order ("global tile index").  Tile t's
 *    num_valid_pages is the number of 128-key blocks up to and including the
 *    block of its last row's position; that last block is its diagonal
 *    block.
 *  - Page table: kv_indices is the flat list of physical page ids, sequence
 *    by sequence, ceil(kv_len/128) entries per sequence (logical block j of
 *    sequence s is page kv_indices[sum_{s'<s} ceil(kv_len_s'/128) + j]).
 *    Page ids must lie in [0, num_pages); a kernel that meets one outside
 *    raises MSA_ERR_DEVICE_CHECK in the plan's error word (read with
 *    msa_check_errors) and skips that block (the appends, and attention over
 *    MSA_KV_FP8_E4M3_BLOCK pages) or reads page 0 in its place (the rest).
 *  - A plan belongs to the device that was current when it was made; its
 *    calls are refused (MSA_ERR_INVALID_ARG) while another one is.
 *  - Errors: host-side argument checks return MSA_ERR_INVALID_ARG or
 *    MSA_ERR_UNSUPPORTED before anything is enqueued; a failed launch
 *    returns MSA_ERR_CUDA.  msa_last_error() gives a message for the
 *    calling thread's last failure.
 *  - NaN inputs are outside the contract and are not scanned for.  A plan
 *    created while the environment variable MSA_CHECKS is set (to anything
 *    but "0") adds, after each of its calls, scans of that call's
 *    floating-point inputs (the query-side arrays q, pq, dout, and the pages
 *    of k/v/pk that kv_indices names; bf16 or e4m3, not the NVFP4 codes, nor
 *    MSA_KV_FP8_E4M3_BLOCK pages, whose unwritten slots may hold any bytes;
 *    the new rows of the appends) and
 *    outputs (max_score, out, lse, dq, dpq, the rows of msa_append_bwd; not
 *    the pages of dk/dv/dpk and of the caches, of which those not referenced
 *    keep the caller's contents), and raises MSA_ERR_NONFINITE in the
 *    error word when one holds a NaN.  -inf in max_score and lse is a
 *    defined value (no visible key) and is not flagged.  Each scan is one
 *    read of its array.
 */
#ifndef MSA_H
#define MSA_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream; NULL is the legacy default stream. */
typedef struct CUstream_st* msa_stream_t;

typedef enum {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARG = 1,   /* bad pointer, size or layout */
  MSA_ERR_UNSUPPORTED = 2,   /* valid but outside what the kernels implement */
  MSA_ERR_CUDA = 3,          /* CUDA runtime / launch failure */
  MSA_ERR_NO_MEMORY = 4,     /* plan workspace allocation failed */
  MSA_ERR_TIMEOUT = 5,       /* a bounded device-side wait gave up */
  MSA_ERR_DEVICE_CHECK = 6,  /* a device-side bounds check fired (bad page id) */
  MSA_ERR_NONFINITE = 7      /* MSA_CHECKS: a NaN reached an output */
} msa_status;

typedef enum {
  MSA_KV_BF16 = 0,           /* K/V pages are bfloat16 */
  MSA_KV_FP8_E4M3 = 1,       /* K/V pages are OCP e4m3 with one fp32 scale per KV head */
  MSA_KV_FP8_E4M3_BLOCK = 2  /* K/V pages are OCP e4m3 with one fp32 scale per (page, KV head) */
} msa_kv_dtype;

typedef enum {
  MSA_BF16 = 0,
  MSA_F32 = 1
} msa_dtype;

typedef enum {
  MSA_ROPE_HALF = 0,         /* pairs (i, i + rotary_dim / 2) */
  MSA_ROPE_INTERLEAVED = 1   /* pairs (2 i, 2 i + 1) */
} msa_rope_layout;

typedef enum {
  MSA_ROPE_NONE = 0,
  MSA_ROPE_LINEAR = 1,       /* positions divided by the factor */
  MSA_ROPE_NTK = 2,          /* base * factor^(rotary_dim / (rotary_dim - 2)) */
  MSA_ROPE_YARN = 3          /* by parts, with the factor on the rotated values */
} msa_rope_scaling;

typedef struct msa_plan_s* msa_plan_t;
typedef struct msa_rope_s* msa_rope_t;

/*
 * msa_plan -- validate a batch shape and build the device tables every
 * other call reads ([README] "Usage": fmha_sm100_plan(qo_lens, kv_lens,
 * heads, num_kv_heads, page_size, kv_block_num=topk)).
 *
 *  qo_lens, kv_lens  HOST int32[batch]; 0 <= qo_lens[s] <= kv_lens[s],
 *                    kv_lens[s] >= 1, and at least one qo_lens[s] > 0 (a
 *                    sequence with qo_len 0 has no tiles; its pages keep
 *                    their page-table entries).  Otherwise
 *                    MSA_ERR_INVALID_ARG.  Copied; the caller keeps
 *                    ownership.
 *  num_qo_heads      Hq, query heads of the main attention.
 *  num_kv_heads      Hkv, KV heads (GQA groups); Hq % Hkv == 0.
 *  num_proxy_heads   Hp, proxy query heads, a multiple of Hkv that divides
 *                    Hq ([FLASH]: at least one proxy head per GQA group,
 *                    each with its own block set).  Proxy head p serves
 *                    query heads [p*Hq/Hp, (p+1)*Hq/Hp), all of KV head
 *                    p / (Hp/Hkv): with Hp = Hkv that is one proxy head per
 *                    GQA group; with Hp = m*Hkv each group's query heads
 *                    split into m sets with a block set each.
 *  head_dim          d in {64, 128}.
 *  proxy_head_dim    dp in {32, 64}.
 *  page_size         must be 128 ([README] "page_size, topk = 128, 16").
 *  topk              K >= 1 selected blocks per (tile, proxy head), the
 *                    diagonal block included.
 *  num_pages         physical pages in the K/V page pool (and the proxy K
 *                    pool, which shares page ids); at most 2^24, and so
 *                    num_pages * Hkv with MSA_KV_FP8_E4M3_BLOCK.
 *  kv_dtype          element type of k_pages / v_pages.
 *  flags             reserved, pass 0.
 *  stream            stream for the one host->device copy of the tables.
 *  out               receives the plan; release with msa_plan_destroy.
 *
 * Allocates the plan's device tables and workspace (this is the only call
 * that allocates) and waits for their upload.
 */
msa_status msa_plan(const int32_t* qo_lens, const int32_t* kv_lens, int32_t batch,
                    int32_t num_qo_heads, int32_t num_kv_heads, int32_t num_proxy_heads,
                    int32_t head_dim, int32_t proxy_head_dim, int32_t page_size, int32_t topk,
                    int64_t num_pages, msa_kv_dtype kv_dtype, uint32_t flags,
                    msa_stream_t stream, msa_plan_t* out);

void msa_plan_destroy(msa_plan_t plan);

/* Shape queries of a plan. */
int32_t msa_plan_num_tiles(msa_plan_t plan);     /* tiles across the batch */
int32_t msa_plan_max_blocks(msa_plan_t plan);    /* max_s ceil(kv_len_s/128) */
int64_t msa_plan_total_q(msa_plan_t plan);       /* sum of qo_lens */
/* DEVICE int32[num_tiles]: num_valid_pages per tile (owned by the plan). */
const int32_t* msa_plan_num_valid_pages(msa_plan_t plan);

/*
 * msa_proxy_maxscore -- stage 1, the proxy pass ([README] "Usage": dense
 * proxy pass with output_o=False, output_maxscore=True; [FLASH]: blocks of
 * 128 tokens chosen by max-pooling over proxy scores).
 *
 *   max_score[t, h, j] = max over rows i of tile t and keys k of block j
 *                        with k visible to i of  pq[i,h] . pk[k] / sqrt(dp)
 *                        (-inf where no pair is visible, and for j beyond
 *                        the tile's num_valid_pages).
 *
 *  pq         bf16 [total_q, Hp, dp].
 *  pk_pages   bf16 [num_pages, 1, 128, dp]: one shared proxy K head, paged
 *             with the same kv_indices as the main K/V.
 *  kv_indices int32 page table (see conventions).
 *  max_score  fp32 [num_tiles, Hp, max_blocks], written entirely.
 * The proxy V of the reference call is not taken: nothing reads it when no
 * output O is produced.
 */
msa_status msa_proxy_maxscore(msa_plan_t plan, const void* pq, const void* pk_pages,
                              const int32_t* kv_indices, float* max_score, msa_stream_t stream);

/*
 * msa_proxy_maxscore_fp8 -- stage 1 at decode with the proxy K stored as
 * FP8 e4m3 ("MiniMax-AI/MSA" README, section "Stacks": the FP8 paged decode
 * stack; an FP8 proxy K halves the proxy scan, which is the largest read of
 * a decode step).  The logit of a pair is (pq[i,h] . pk_code[k]) *
 * pk_scale[0] / sqrt(dp), the same dequantisation as the FP8 main K;
 * otherwise max_score is defined as in msa_proxy_maxscore.
 *
 *  pq         bf16 [total_q, Hp, dp].
 *  pk_pages   e4m3 codes [num_pages, 1, 128, dp], 16-byte aligned.
 *  pk_scale   device pointer to one fp32 scale (> 0) for the shared proxy head.
 * Plans whose sequences all have qo_len = 1, dp = 64 and Hp <= 8 only;
 * others return MSA_ERR_UNSUPPORTED.
 */
msa_status msa_proxy_maxscore_fp8(msa_plan_t plan, const void* pq, const void* pk_pages,
                                  const float* pk_scale, const int32_t* kv_indices, float* max_score,
                                  msa_stream_t stream);

/*
 * msa_proxy_maxscore_nvfp4 -- stage 1 at decode with the proxy K stored in
 * NVFP4, the FP4 block-score indexer ("MiniMax-AI/MSA" README, section
 * "Stacks": the FP4 block-score indexer; Flash-MSA article, "what's next":
 * the indexer in low precision).  The shared proxy head's keys are e2m1
 * codes with one e4m3 scale per 16 consecutive dimensions and one fp32
 * scale for the head:
 *   pk[k, d] = e2m1(code[k, d]) * e4m3(block_scale[k, d / 16]) * global_scale
 * and the logit of a pair is pq[i,h] . pk[k] / sqrt(dp); otherwise max_score
 * is defined as in msa_proxy_maxscore.  The proxy K read is a quarter of the
 * bf16 one (plus 1/8 for the scales).
 *
 *  pq               bf16 [total_q, Hp, dp].
 *  pk_codes         uint8 [num_pages, 1, 128, dp / 2], 16-byte aligned: byte
 *                   b of a key holds dims 2b (low nibble) and 2b + 1 (high
 *                   nibble), each e2m1 (1 sign, 2 exponent bits with bias 1,
 *                   1 mantissa bit; exponent 0 is 0 or 0.5).
 *  pk_block_scales  e4m3 [num_pages, 1, 128, dp / 16], 16-byte aligned.
 *  pk_global_scale  device pointer to one fp32 scale (> 0).
 * Decode plans (every qo_len == 1) with dp = 64 and Hp <= 8 only; others
 * return MSA_ERR_UNSUPPORTED.  The products run on f16 tensor cores with pq
 * rounded to f16 (exact for |pq| in [2^-14, 65504]); code * block scale is
 * exact in f16.
 */
msa_status msa_proxy_maxscore_nvfp4(msa_plan_t plan, const void* pq, const void* pk_codes,
                                    const void* pk_block_scales, const float* pk_global_scale,
                                    const int32_t* kv_indices, float* max_score, msa_stream_t stream);

/*
 * msa_topk_select -- stage 2 ([README] sparse_topk_select(max_score, topk,
 * num_valid_pages); [FLASH]: each proxy head picks its own block set, the
 * local block is always visible).  Plan-free, like the reference call.
 *
 * For each row (t, h) with n = num_valid_pages[t] and diagonal block
 * j_d = n - 1: if topk >= n the row selects blocks 0..n-1; otherwise it
 * selects j_d plus the topk-1 largest max_score[t,h,j] over j < j_d,
 * ignoring -inf, ordered by (score descending, j ascending); -0.0 and +0.0
 * are equal.  Selected indexes are written ascending, padded with -1.
 * Scores are compared exactly (bit-exact result); NaN inputs are outside
 * the contract.
 *
 *  max_score        fp32 [n_tiles, heads, max_blocks].
 *  num_valid_pages  int32 [n_tiles], each in [1, max_blocks].  A row whose
 *                   value lies outside that range selects nothing: it is
 *                   written as topk entries of -1 (the attention then
 *                   treats its query rows as seeing no key).
 *  kv_block_indexes int32 [n_tiles, heads, topk] (output).
 *  1 <= topk <= 1024, max_blocks <= 65536.
 */
msa_status msa_topk_select(const float* max_score, int32_t n_tiles, int32_t heads,
                           int32_t max_blocks, int32_t topk, const int32_t* num_valid_pages,
                           int32_t* kv_block_indexes, msa_stream_t stream);

/*
 * msa_proxy_topk -- stages 1 and 2 fused ([FLASH], kernel-design
 * paragraph: the forward proxy pass keeps a streaming top-k over blocks in
 * registers instead of accumulating outputs).  The proxy pass and the
 * selection of msa_proxy_maxscore + msa_topk_select in one launch, with no
 * max_score round trip.
 *
 * Writes the same kv_block_indexes as msa_topk_select(max_score, ...,
 * plan topk, msa_plan_num_valid_pages(plan), ...) would on the scores that
 * msa_proxy_maxscore writes: bit-exact, ties to the lower block, ascending,
 * -1 padded.  The work units of one tile report their candidates and the
 * last of them merges; nothing waits on another CTA.
 *
 *  pq, pk_pages, kv_indices  as for msa_proxy_maxscore.
 *  max_score         fp32 [num_tiles, Hp, max_blocks] (output) or NULL.
 *  kv_block_indexes  int32 [num_tiles, Hp, topk] (output).
 * Prefill plans with topk <= 32 and at most 1024 blocks per sequence;
 * others return MSA_ERR_UNSUPPORTED (use the two separate calls).  The
 * plan's counters are reset by every complete launch, so two calls on one
 * plan must not overlap in time; after a launch that failed with a device
 * error the plan must be rebuilt.
 */
msa_status msa_proxy_topk(msa_plan_t plan, const void* pq, const void* pk_pages,
                          const int32_t* kv_indices, float* max_score, int32_t* kv_block_indexes,
                          msa_stream_t stream);

/*
 * msa_sparse_attn -- stage 3, GQA block-sparse attention forward ([README]
 * "Usage": fmha_sm100(q, k_pages, v_pages, sparse_plan, kv_indices,
 * kv_block_indexes); [STACKS]: paged FP8 decode; [FLASH]: GQA main
 * attention over the selected blocks).
 *
 * For query row i of tile t and head h (KV head g = h / (Hq/Hkv), proxy
 * head p = h / (Hq/Hp)): softmax over the keys k of KV head g in blocks
 * kv_block_indexes[t, p, :] (entries < 0 are skipped) with k visible to i
 * of s = q[i,h].k[k] / sqrt(d); out = P.V, lse = natural-log logsumexp of
 * s.  With FP8 K/V: s uses k*k_scale[g] and V is v*v_scale[g]
 * ([STACKS]: FP8 for the paged decode and the sparse prefill).
 *
 *  q                 bf16 [total_q, Hq, d].
 *  k_pages, v_pages  [num_pages, Hkv, 128, d], bf16 or e4m3 per the plan
 *                    (MSA_KV_FP8_E4M3: head_dim 128, at decode at most 16
 *                    query heads per proxy head; the e4m3 MMAs run in f16, with
 *                    q rounded to f16, exact for |q| in [2^-14, 65504] and
 *                    saturating beyond).
 *  kv_indices        int32 page table.
 *  kv_block_indexes  int32 [num_tiles, Hp, topk], as msa_topk_select writes
 *                    them.  Any order of distinct valid blocks is accepted,
 *                    with -1 entries anywhere.  In prefill a query row that
 *                    sees no key of its selection gets out = 0 and
 *                    lse = -inf (a row of only -1 included); decode
 *                    selections must hold the diagonal (last) block.
 *  k_scale, v_scale  fp32 [Hkv] for MSA_KV_FP8_E4M3, fp32 [num_pages, Hkv]
 *                    for MSA_KV_FP8_E4M3_BLOCK, NULL for bf16.
 *  out               bf16 [total_q, Hq, d] (output).
 *  lse               fp32 [total_q, Hq] (output) or NULL.
 * MSA_KV_FP8_E4M3_BLOCK: s uses k * k_scale[page, g] and V is v *
 * v_scale[page, g] of the page that holds the key.  Scales are taken as lying in
 * [2^-40, 2^40] (others, zero and NaN among them, count as the nearer end).
 * Slots of a sequence's last page behind its last key may hold any bytes.  At
 * decode, too, a row that sees no key of its selection gets out = 0 and
 * lse = -inf.  These plans use no workspace: their calls may overlap.
 *
 * Decode batches (every qo_len == 1) run a split-K kernel whose partial
 * results live in the plan's workspace: two calls on one plan must not
 * overlap in time (issue them on one stream, or order the streams).
 */
msa_status msa_sparse_attn(msa_plan_t plan, const void* q, const void* k_pages, const void* v_pages,
                           const int32_t* kv_indices, const int32_t* kv_block_indexes,
                           const float* k_scale, const float* v_scale,
                           void* out, float* lse, msa_stream_t stream);

/*
 * msa_sparse_attn_bwd -- training extension: the fused backward ([FLASH]
 * backward-pass paragraph: the KL between the proxy and main attention
 * distributions needs both, so both gradients come from one pass; the KL
 * gradient with respect to a proxy logit is p_proxy - p_main; block indexes
 * are the ones cached from the forward).
 *
 * Main part, restricted to the cached blocks and the causal mask, for the
 * scalar sum(out * dout):  D = rowsum(dout*out), dS = P*(dP - D),
 * dq = dS.K/sqrt(d), dk = dS^T.q/sqrt(d) and dv = P^T.dout summed over the
 * heads (and selections) of a KV head.  KL part, per row i and proxy head p
 * over the same keys as p's query heads: p_main = mean of the P of the
 * Hq/Hp heads that use p's blocks (no gradient), p_proxy = softmax of
 * pq[i,p].pk/sqrt(dp), dZ = kl_weight*(p_proxy - p_main), dpq =
 * dZ.pk/sqrt(dp), dpk = dZ^T.pq/sqrt(dp).  A page named by several
 * page-table entries (a shared prefix) gets the sum over all of them in
 * dk_pages, dv_pages and dpk_pages.  Rows that see no key of their
 * selection get dq = 0 and dpq = 0 and add nothing elsewhere.
 *
 *  q, k_pages, v_pages, kv_indices, kv_block_indexes  as in the forward
 *                    (bf16 K/V only).
 *  out, lse          the forward's bf16 out and fp32 lse.
 *  dout              bf16 [total_q, Hq, d].
 *  pq, pk_pages      the proxy inputs of msa_proxy_maxscore.
 *  dq                fp32 [total_q, Hq, d]            (output, overwritten)
 *  dk_pages,dv_pages fp32 [num_pages, Hkv, 128, d]    (output; pages the
 *                    plan's sequences reference are overwritten, others
 *                    untouched)
 *  dpq               fp32 [total_q, Hp, dp]           (output, overwritten)
 *  dpk_pages         fp32 [num_pages, 1, 128, dp]     (output, as dk_pages)
 * q, k_pages, v_pages, out, dout, pq and pk_pages must be 16-byte aligned and
 * the five gradients 32-byte aligned (MSA_ERR_INVALID_ARG otherwise).
 */
msa_status msa_sparse_attn_bwd(msa_plan_t plan, const void* q, const void* k_pages,
                               const void* v_pages, const int32_t* kv_indices,
                               const int32_t* kv_block_indexes, const void* out, const float* lse,
                               const void* dout, const void* pq, const void* pk_pages,
                               float kl_weight, float* dq, float* dk_pages, float* dv_pages,
                               float* dpq, float* dpk_pages, msa_stream_t stream);

/*
 * msa_sparse_decode_noalloc -- the FP8 paged decode of msa_sparse_attn for
 * callers that cannot allocate device memory when they decode (for example
 * a server that gives the GPU's memory to its own pool at start-up, or a
 * decode loop that must not pay for cudaMalloc's implicit synchronisation;
 * neither can create a plan, since msa_plan allocates).  The paper has no
 * counterpart: this is a deployment variant of the decode kernel.
 *
 * Computes exactly what msa_sparse_attn computes for a decode batch (one
 * query row per sequence) with e4m3 K/V, head_dim 128, up to 16 query heads
 * per KV head.  The batch comes as DEVICE arrays instead of a plan:
 *   kv_lens    int32 [batch], keys per sequence (>= 1);
 *   kv_indptr  int32 [batch+1], offset of each sequence's pages in
 *              kv_indices (kv_indptr[s+1] - kv_indptr[s] >= ceil(kv_len/128)).
 * q, k_pages, v_pages, kv_indices, kv_block_indexes ([batch, Hkv, topk]),
 * k_scale, v_scale, out and lse (nullable) are as in msa_sparse_attn.
 * err_word: optional DEVICE uint32 that the kernels OR status bits into;
 * NULL discards them.  Bit 0: a device-side bounds check fired (a bad page
 * id or page range; that block is skipped or read from page 0).  Bit 1: a
 * bounded device-side wait gave up; the call's out and lse are then
 * unspecified.  The caller clears the word.
 *
 * Scratch: all of it (a tile table and the split-K partials) lives in one
 * fixed 24 MiB device array inside libmsa, held by every GPU that loads the
 * library until the process exits.  The call allocates nothing and calls no
 * allocating routine.  Each call clears the split-K counters of its own rows
 * before using them, so a call that failed does not disturb later ones.  It rejects, with MSA_ERR_INVALID_ARG, batch > 4096 or
 * batch * num_qo_heads * topk above 47,639 (the partials that fit in the
 * array at head_dim 128) or batch * num_kv_heads above 65,536.  The first call on a device looks up the array's
 * device address for that device (cudaGetSymbolAddress) with that device
 * current; make that first call before any stream capture.  Every call on a
 * device shares the one array and overwrites what it needs: calls that
 * overlap on the GPU (other streams, or other host threads) race and give
 * wrong results; issue them one after another.
 */
msa_status msa_sparse_decode_noalloc(const void* q, const void* k_pages, const void* v_pages,
                                     const int32_t* kv_lens, const int32_t* kv_indptr,
                                     const int32_t* kv_indices, const int32_t* kv_block_indexes,
                                     const float* k_scale, const float* v_scale, int32_t batch,
                                     int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t topk, int64_t num_pages, void* out, float* lse,
                                     uint32_t* err_word, msa_stream_t stream);

/*
 * msa_rope_create -- a table of rotary frequencies, for msa_rope_apply and the
 * cache appends.  Pair i of rotary_dim / 2 turns by
 *   f_i = base^(-2 i / rotary_dim)
 * radians a position, and `scaling` stretches that to contexts `factor` times
 * as long:
 *   MSA_ROPE_LINEAR  f_i / factor;
 *   MSA_ROPE_NTK     base * factor^(rotary_dim / (rotary_dim - 2)) for base;
 *   MSA_ROPE_YARN    with D(b) = rotary_dim ln(original_len / (2 pi b)) /
 *                    (2 ln base), lo = max(floor D(beta_fast), 0), hi =
 *                    min(ceil D(beta_slow), rotary_dim - 1) and the ramp
 *                    r_i = clamp((i - lo) / (hi - lo), 0, 1):  (1 - r_i) f_i + r_i f_i / factor,
 *                    and the rotated values are multiplied by m = 0.1 ln
 *                    factor + 1 (m = 1 otherwise).
 *
 *  rotary_dim    a multiple of 16 in [16, 256].
 *  base          above 1.
 *  factor        at least 1; read unless scaling is MSA_ROPE_NONE.
 *  original_len, beta_fast, beta_slow   read for MSA_ROPE_YARN only.
 *  out           receives the handle; release with msa_rope_destroy.
 * Host memory only: the handle serves every device and stream, and calls that
 * were given it keep no reference to it (they copy the table at the launch).
 * Angles are right to fp32 at every int32 position: the table has 64-bit
 * fractions of a turn, and the phase is an integer product modulo one turn.
 */
msa_status msa_rope_create(int32_t rotary_dim, msa_rope_layout layout, double base, msa_rope_scaling scaling,
                           double factor, int32_t original_len, double beta_fast, double beta_slow,
                           msa_rope_t* out);

void msa_rope_destroy(msa_rope_t rope);

/*
 * msa_rope_apply -- rotary positions: with t = f_i * positions[row] and (a, b)
 * pair i of a head,  a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t);
 * dims from rotary_dim on are copied.  With inverse != 0 the rotation is by
 * -t (and still times m): the transpose, which takes the gradient of the
 * rotated heads to that of the heads.  cos, sin (times m), the products and
 * their sum are rounded in fp32 each, as elementwise arithmetic rounds them; a
 * bf16 result once more.
 *
 *  x             bf16 or fp32 [n_rows, heads, head_dim]; rows x_row_stride
 *                elements apart, heads dense within a row (a slice of a fused
 *                projection's rows serves).
 *  positions     int32 [n_rows], any values.
 *  n_rows        >= 0 (0: nothing is done).
 *  head_dim      a multiple of 16 up to 256, at least rotary_dim.
 *  out           as x, rows out_row_stride elements apart; x itself (in
 *                place) or memory that shares no row with it.
 * Rows must start on 16-byte boundaries (MSA_ERR_INVALID_ARG otherwise).
 */
msa_status msa_rope_apply(msa_rope_t rope, const void* x, int64_t x_row_stride, const int32_t* positions,
                          int64_t n_rows, int32_t heads, int32_t head_dim, msa_dtype dtype, int32_t inverse,
                          void* out, int64_t out_row_stride, msa_stream_t stream);

/*
 * msa_kv_append -- writes a batch's new K and V rows into the paged cache that
 * msa_sparse_attn reads: row r of a sequence, at key position kv_len - qo_len
 * + r, goes to slot position % 128 of the page of its block.  K is rotated
 * first when a rope is given.
 *
 *  rope          NULL: K is written as it is.
 *  positions     int32 [total_q] for the rotation, or NULL for the key
 *                positions.
 *  k, v          bf16 [total_q, Hkv, d], rows k_row_stride / v_row_stride
 *                elements apart, each starting on a 16-byte boundary.
 *  kv_indices    int32 page table.  Pages that get rows must be named once
 *                (a shared prefix ends on a page boundary).
 *  k_pages, v_pages, k_scale, v_scale   the cache, by the plan's kv_dtype:
 *    MSA_KV_BF16            bf16(x); no scales.
 *    MSA_KV_FP8_E4M3        e4m3(x / scale[head]); scale fp32 [Hkv] is read.
 *    MSA_KV_FP8_E4M3_BLOCK  e4m3(x / s), s = scale[page, head], fp32
 *        [num_pages, Hkv], is written: the least power of two s in [2^-40,
 *        2^40] with |x| <= 448 s for the page's new rows (infinities aside),
 *        and not below the page's scale (rounded up to a power of two) when
 *        the rows go behind others on a partly filled page.  Where that
 *        raises the scale, the slots before the new rows are converted to it.
 *        A page whose first slot is written starts anew, whatever scale it
 *        had.  A partly filled page whose scale is not in (0, 2^40] raises
 *        MSA_ERR_DEVICE_CHECK and its old slots keep their bytes; one below
 *        2^-40 counts as 2^-40, as in msa_sparse_attn.
 *    e4m3 conversions are to nearest, ties to even, saturating at +-448.
 * Other slots of the pages keep their contents.  A page id outside the pool is
 * reported (MSA_ERR_DEVICE_CHECK) and its rows are dropped.  One launch; the
 * call uses no workspace of the plan, and appending the same rows again gives
 * the same cache.
 */
msa_status msa_kv_append(msa_plan_t plan, msa_rope_t rope, const int32_t* positions, const void* k,
                         int64_t k_row_stride, const void* v, int64_t v_row_stride, const int32_t* kv_indices,
                         void* k_pages, void* v_pages, float* k_scale, float* v_scale, msa_stream_t stream);

/*
 * msa_pk_append -- writes a batch's new proxy K rows, as msa_kv_append does K,
 * into any of the three pools that the proxy passes read (one at least; a
 * prefill scans bf16, the decode steps after it e4m3 or NVFP4).
 *
 *  pk              bf16 [total_q, dp], rows pk_row_stride elements apart.
 *  pk_pages        bf16 [num_pages, 1, 128, dp], or NULL.
 *  pk_pages_e4m3   e4m3(x / pk_scale[0]), or NULL with pk_scale NULL.
 *  pk_codes, pk_block_scales, pk_global_scale   NVFP4 as
 *                  msa_proxy_maxscore_nvfp4 reads it, or all NULL: the block
 *                  scale is e4m3(amax / (6 g)) over 16 dims, g the global
 *                  scale (read, > 0), and a code e2m1(x / (block scale * g)),
 *                  both to nearest with ties to even, saturating; codes of a
 *                  block whose scale is 0 are 0.
 * rope, positions, kv_indices, errors: as msa_kv_append.
 */
msa_status msa_pk_append(msa_plan_t plan, msa_rope_t rope, const int32_t* positions, const void* pk,
                         int64_t pk_row_stride, const int32_t* kv_indices, void* pk_pages, void* pk_pages_e4m3,
                         const float* pk_scale, void* pk_codes, void* pk_block_scales, const float* pk_global_scale,
                         msa_stream_t stream);

/*
 * msa_append_bwd -- the backward of msa_kv_append and msa_pk_append on bf16
 * plans: the gradients of the new rows out of the gradient pages that
 * msa_sparse_attn_bwd wrote, dK and dpk rotated back (see msa_rope_apply,
 * inverse).
 *
 *  k_rope, pk_rope, positions   as given to the appends (NULL where they were).
 *  dk_pages, dv_pages   fp32 [num_pages, Hkv, 128, d];  dpk_pages fp32
 *                       [num_pages, 1, 128, dp].
 *  dk, dv               fp32 [total_q, Hkv, d];  dpk fp32 [total_q, dp]
 *                       (outputs, overwritten).
 * Each of the three is left out with both its pointers NULL.  All must be
 * 16-byte aligned.  Rows of a page id outside the pool are zero, and
 * reported.
 */
msa_status msa_append_bwd(msa_plan_t plan, msa_rope_t k_rope, msa_rope_t pk_rope, const int32_t* positions,
                          const int32_t* kv_indices, const float* dk_pages, const float* dv_pages,
                          const float* dpk_pages, float* dk, float* dv, float* dpk, msa_stream_t stream);

/*
 * msa_check_errors -- waits for `stream`, then reads and clears the plan's
 * device error word: MSA_OK, MSA_ERR_TIMEOUT (a bounded wait inside a kernel
 * gave up; that kernel's outputs are unspecified), MSA_ERR_DEVICE_CHECK (a
 * kernel met a page id or a block out of range) or, for plans
 * created under MSA_CHECKS, MSA_ERR_NONFINITE (an output held a NaN), in
 * that order when several are set.
 */
msa_status msa_check_errors(msa_plan_t plan, msa_stream_t stream);

/*
 * msa_selftest_wait_timeout -- the failure-detection path, on the device:
 * launches one kernel whose bounded mbarrier wait cannot complete (nothing
 * arrives on the barrier).  The wait gives up after its 2 s limit, the
 * kernel records the timeout in an error word and returns, the context stays
 * usable, and the call reports what msa_check_errors reports for any kernel
 * whose wait ran out: MSA_ERR_TIMEOUT.  Any other error word gives
 * MSA_ERR_CUDA.  Synchronises `stream`; allocates and frees 4 bytes.
 */
msa_status msa_selftest_wait_timeout(msa_stream_t stream);

/*
 * msa_test_fail_plan_allocs -- failure injection on the host, for tests of a
 * caller's out-of-memory handling: the next `count` calls of msa_plan that
 * reach their device allocation fail there exactly as a failed cudaMalloc
 * does (MSA_ERR_NO_MEMORY, nothing allocated, *out left NULL), without
 * calling cudaMalloc.  count <= 0 cancels what is left.  Process-wide.
 */
void msa_test_fail_plan_allocs(int32_t count);

/* Message for the calling thread's last failed call ("" if none). */
const char* msa_last_error(void);

/* Library version, "major.minor.patch". */
const char* msa_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MSA_H */
