/* Kernel-level entry points of the PCD library: single device steps, for
 * testing them in isolation against the CPU oracle, and the operators of a
 * serving layer (rotary positions, an 8-bit paged cache, attention over it).
 * Every pointer is a DEVICE pointer the caller owns; nothing is allocated or freed here.  Each call is enqueued on
 * `stream` (a cudaStream_t, NULL = legacy default stream) and returns without
 * synchronising.  Return value: 0 on success, a negative PCD_ERR_* code
 * (pcd.h) for invalid arguments, or PCD_ERR_CUDA when the launch fails.
 */
#ifndef PCD_KERNELS_H
#define PCD_KERNELS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Epilogue kinds of pcd_k_gemm. */
#define PCD_EPI_BF16 0       /* out fp16 [M][ldo] = A.B^T (16-bit store)                    */
#define PCD_EPI_F32_ADD 1    /* out f32 [M][ldo] += A.B^T (splits must be 1)                */
#define PCD_EPI_F32_ATOMIC 2 /* out f32 [M][ldo] += A.B^T with atomics (any splits)         */
#define PCD_EPI_SWIGLU 3     /* out fp16 [M][ldo]: col f = silu(D[:,2f]) * D[:,2f+1]        */

/* Dense projection on the tensor cores: D[M][N] = A[M][K] . B[N][K]^T with
 * fp16 A and B (row-major, K contiguous, leading dimensions lda/ldb in
 * elements, multiples of 8), fp32 accumulation and a fused epilogue.  This is
 * the contraction of every QKV, output and SwiGLU projection of the decoder
 * (configs: nn.Linear weights [out][in] as B, activations [tokens][in] as A).
 * K must be a multiple of 64, N a multiple of 32.  mt/bn/splits force a
 * tiling (mt in {1,2,4}, bn in {128,256}); mt = 0 lets the library choose;
 * mt = 3 runs CTA pairs that share one tensor-core MMA of 256 rows (each CTA
 * loads its 128 rows of A and half of the B tile).
 * `dev_err` (device int, may be NULL) receives a nonzero code if a pipeline
 * wait times out. */
int pcd_k_gemm(const void* a, int M, int lda, const void* b, int N, int ldb, int K, int epi, void* out, int ldo,
               int mt, int bn, int splits, int* dev_err, void* stream);

/* pcd_k_gemm with A given as two fp16 halves, a_hi + a_lo (a_lo the rounding
 * remainder of an fp32 activation): D = (A_hi + A_lo) . B^T, both products
 * accumulated in one fp32 accumulator from one read of B.  One 128-row tile
 * per CTA; epi PCD_EPI_F32_ADD, PCD_EPI_F32_ATOMIC or PCD_EPI_SWIGLU; bn in
 * {128, 256}. */
int pcd_k_gemm_split(const void* a_hi, const void* a_lo, int M, int lda, const void* b, int N, int ldb, int K, int epi,
                     void* out, int ldo, int bn, int splits, int* dev_err, void* stream);

/* pcd_k_gemm in the weight-streaming form for short activations (M <= 512
 * token rows: the branch rows of one request, How TypeSafe's Jev Might Work,
 * "One forward pass for all fields"): the same D[M][N] = (A + A_lo)[M][K] .
 * B[N][K]^T, computed with B (the weights) as the 256-row side of a tensor-core
 * MMA shared by a pair of CTAs and A as its N side, so every weight tile is
 * read from HBM once.  a_lo (may be NULL) is A's fp16 rounding remainder.
 * epi PCD_EPI_F32_ADD (splits 1), PCD_EPI_F32_ATOMIC (splits >= 1; 0 lets the
 * library choose) or PCD_EPI_SWIGLU (splits 1; B rows 2f, 2f+1 are gate f and
 * up f, out[M][ldo] fp16).  K a multiple of 64, N a multiple of 32, lda/ldb
 * multiples of 8.  Returns 0, -1 for an invalid shape, -10 for a launch
 * error; `dev_err` as in pcd_k_gemm. */
int pcd_k_gemm_swap(const void* a, const void* a_lo, int M, int lda, const void* b, int N, int ldb, int K, int epi,
                    void* out, int ldo, int splits, int* dev_err, void* stream);

/* Fused vocabulary readout: the LM-head contraction z = h . W^T run tile by
 * tile on the tensor cores with an online log-sum-exp over the whole
 * vocabulary and a gather of selected logits, so the [R][V] logits are never
 * written (PCD: A Technical Reference, section 4, stages 3-4: read only the
 * candidate logits; the log-sum-exp turns them into full-vocabulary
 * log-probs).  h [R][d] and w [V][d] are fp16 device matrices (K
 * contiguous, d a multiple of 64, V a multiple of 32).  The gathered pairs are
 * HOST arrays cand_row/cand_tok[n_cand] (row < R, token < V).  Outputs
 * (device): lse[R] = log sum_v exp(z[r][v]) and z_out[n_cand] =
 * z[cand_row][cand_tok], fp32.  `scratch` is a device buffer of at least
 * pcd_k_readout_scratch_bytes(R, V, n_cand) bytes that the call overwrites
 * (per-tile partial maxima and sums, the tile-sorted gather list).  Enqueued
 * on `stream`; the gather list is copied from host memory first, from a
 * buffer that lives only until the call returns, so a call made while
 * `stream` is being captured into a CUDA graph returns PCD_ERR_INVALID_ARG
 * without enqueueing anything. */
int64_t pcd_k_readout_scratch_bytes(int R, int V, int n_cand);
int pcd_k_readout(const void* h, int R, const void* w, int V, int d, const int32_t* cand_row, const int32_t* cand_tok,
                  int n_cand, float* lse, float* z_out, void* scratch, int64_t scratch_bytes, int* dev_err,
                  void* stream);

/* pcd_k_readout without a scratch argument, for callers that cannot allocate
 * device memory: a serving loop whose GPU memory is already reserved by its
 * own pool (a fresh cudaMalloc would fail or fragment it), or code on a
 * latency-critical stream where cudaMalloc / cudaFree would synchronise the
 * device and stall every other stream.  (The pages have no counterpart: it is
 * a property of this library's interface, not of the method.)
 * The scratch is one file-scope __device__ array of
 * PCD_K_READOUT_NOALLOC_MAX_BYTES bytes that every GPU loading the library
 * holds until the process exits.  Inputs, outputs and errors are those of
 * pcd_k_readout; a problem whose pcd_k_readout_scratch_bytes(R, V, n_cand)
 * exceeds the array returns PCD_ERR_OOM without launching anything.  Every
 * call looks up the array's device address (cudaGetSymbolAddress) with the
 * caller's device current; the first call on a device also loads the
 * library's device code there, so make that first call before any stream
 * capture.  No call allocates or frees memory.  Every call
 * shares the one array and leaves its contents behind; each call writes every
 * scratch element it reads before reading it, so nothing needs clearing, but
 * calls that overlap on the GPU (other streams, other threads) race on the
 * array and must be serialised by the caller. */
#define PCD_K_READOUT_NOALLOC_MAX_BYTES (8 * 1024 * 1024)
int pcd_k_readout_noalloc(const void* h, int R, const void* w, int V, int d, const int32_t* cand_row,
                          const int32_t* cand_tok, int n_cand, float* lse, float* z_out, int* dev_err, void* stream);

/* Bounded-wait check (the pages have no counterpart: it exercises this
 * library's failure path, a pipeline partner that never arrives, without
 * faulting or hanging the GPU).  One thread waits on a shared-memory mbarrier
 * that nothing ever arrives on, with the bounded wait every pipeline of the
 * library uses, and gives up once `limit_ns` (0 .. 10^10) has passed: it
 * then records a nonzero code in `dev_err` (a device int, which it never
 * clears) and writes the wait's duration in ns, by the device's global timer,
 * to `elapsed_ns` (a device int64, may be NULL).  Enqueued on `stream`;
 * returns 0, -1 for a bad argument (nothing enqueued) or -10 for a launch
 * error. */
int pcd_k_wait_probe(int64_t limit_ns, int* dev_err, int64_t* elapsed_ns, void* stream);

/* Host-only view of the branch compiler (no GPU needed): compiles `fields`
 * (pcd.h) for a vocabulary of `vocab` tokens into the packed branch batch the
 * branch pass runs (How TypeSafe's Jev Might Work, "When one token is not
 * enough": scaffold tokens plus every internal node of the label trie).
 * sizes[0..7] receives T (branch tokens), R (readout rows), C (child
 * entries), NL (candidate paths), NP (path steps), NA (ancestor entries),
 * NF (fields), NO (labels the paths spell).  When `arrays` is non-NULL,
 * arrays[i] (caller-allocated, sized from a first call with arrays == NULL;
 * a NULL entry is skipped) receives:
 *  0 tok[T], 1 rel[T] (position after the prefix end), 2 anc_off[T+1],
 *  3 anc_idx[NA] (ancestors of each token, itself included, same field),
 *  4 ro_tok[R] (branch token read at each readout row), 5 row_ch[R+1],
 *  6 ch_tok[C] (candidate next token of each child entry), 7 child_row[C],
 *  8 lab_off[NL+1], 9 path[NP] (child entry of each step of each label),
 *  10 fld_lab[NF+1], 11 fld_root[NF] (readout row of each scaffold end),
 *  12 cand_label[NL] (label, within its field, each path spells),
 *  13 fld_out[NF+1] (labels of each field), 14 scoring[NF] (PCD_SCORE_*).
 * ctx[0..n_ctx) (NULL / 0 for none): context tokens written before every
 * field (first field first's answer line), compiled as the first branch
 * tokens.  Returns 0 or the PCD_ERR_* validation code pcd_score would return. */
int pcd_plan_inspect(const void* fields, int n_fields, int vocab, int32_t* sizes, int32_t* const* arrays,
                     const int32_t* ctx, int n_ctx);

/* Host only, no GPU: the answer line first field first writes for `field`
 * (a pcd_field, pcd.h) decided as `label`: its scaffold, the first listed
 * candidate path that spells the label, then sep[0..n_sep) (How TypeSafe's
 * Jev Might Work, "The first key of a JSON object is a special position").
 * Writes at most cap tokens to out (may be NULL with cap = 0) and returns the
 * line's length, or PCD_ERR_INVALID_ARG when no path spells the label. */
int pcd_answer_line(const void* field, int label, const int32_t* sep, int n_sep, int32_t* out, int cap);

/* ------------------------------------------------- rotary positions, paged cache
 * The calls below serve many requests over one pool of cache pages, beside
 * the contiguous caches of pcd.h: rotate the queries (pcd_k_rope), store the
 * new keys and values (pcd_k_kv_append), attend (pcd_k_paged_attention).  They
 * follow the conventions above: device pointers, no allocation, no
 * synchronisation, and they may be captured into CUDA graphs.  What they find
 * wrong in device arrays (offsets, lengths, pages out of range) is skipped
 * and recorded as a nonzero code in `dev_err` (device int, may be NULL).  So is
 * a wait inside pcd_k_paged_attention's pipelines that runs out (2 s, or the
 * PCD_WAIT_LIMIT_MS of the process's first call); the rows it should have
 * computed are then NaN, and their log-sum-exp too.
 * pcd_last_error() says why a call was refused. */
#define PCD_DTYPE_F16 3 /* beside PCD_DTYPE_F32 and PCD_DTYPE_BF16 of pcd.h */

/* Frequencies of rotary positions.  Pair i of the rot_dim / 2 pairs turns by
 * f_i = theta^(-2i / rot_dim) radians a position, changed for contexts longer
 * than the trained orig_len by
 *   PCD_ROPE_LINEAR  f_i / factor;
 *   PCD_ROPE_BASE    theta grown by factor^(rot_dim / (rot_dim - 2));
 *   PCD_ROPE_BANDS   pairs that turn at least hi_turns times over orig_len
 *                    stay, those under lo_turns are divided by factor, a
 *                    blend linear in their turns between;
 *   PCD_ROPE_RAMP    the same ends with a ramp linear in the pair's index,
 *                    between the indices where pairs turn hi_turns and
 *                    lo_turns times (rounded outwards); cos and sin are
 *                    multiplied by 0.1 ln(factor) + 1.
 * factor >= 1; orig_len and the turns are read by the last two only.  Writes
 * rot_dim / 2 HOST values: f_i as a fraction of a turn in units of 2^-64, so
 * that a position's angle is one wrapping integer product, exact at any int32
 * position; the caller copies them to the device.  `amp` (may be NULL)
 * receives the factor on cos and sin. */
#define PCD_ROPE_NONE 0
#define PCD_ROPE_LINEAR 1
#define PCD_ROPE_BASE 2
#define PCD_ROPE_BANDS 3
#define PCD_ROPE_RAMP 4
int pcd_rope_freqs(int rot_dim, double theta, int scaling, double factor, double orig_len, double lo_turns,
                   double hi_turns, int64_t* freqs, float* amp);

/* Rotates the first rot_dim channels of every head of x [n_tok][heads]
 * [head_dim] into y (the other channels are copied; rot_dim 0 with freqs NULL
 * copies all).  dtype: PCD_DTYPE_F32, _F16 or _BF16 for both; arithmetic in
 * fp32, one rounding.  Strides of tokens and heads in elements, channels
 * contiguous.  Pair (a, b) at angle phi becomes amp (a cos phi - b sin phi,
 * b cos phi + a sin phi); pairs are channels (2i, 2i + 1) when `interleaved`,
 * else (i, i + rot_dim / 2).  transpose != 0 turns by -phi with the same amp:
 * the gradient of the rotation.  Token t is at pos[t], or base + t when pos is
 * NULL; any int32 pos and base, negative ones included (base + t may pass
 * 2^31).  y may be x's own view; another overlap is refused, as are strides that
 * put two rows of y in one place and n_tok * head_dim of 2^31 and more. */
int pcd_k_rope(const void* x, void* y, int dtype, int n_tok, int heads, int head_dim, int64_t x_tok, int64_t x_head,
               int64_t y_tok, int64_t y_head, const int64_t* freqs, int rot_dim, int interleaved, float amp,
               const int32_t* pos, int base, int transpose, void* stream);

/* A pool of cache pages in 8 bits.  The K and V codes of (page, KV head, slot)
 * are head_dim bytes at page * page_stride + head * head_stride + slot *
 * token_stride of `k` and `v` (strides and bases multiples of 16 bytes,
 * token_stride at most 2^24), so both [page][head][slot] and
 * [page][slot][head] orders serve.  A page holds page_size (16, 32, 64 or
 * 128) consecutive tokens of one sequence; each (page, KV head) has one scale
 * in k_scale / v_scale [n_pages][n_kv_heads], fp32: value = code * scale.
 * head_dim 64 or 128. */
#define PCD_KV_E4M3 1 /* 8-bit floats, 4 exponent bits; scales are powers of two when written here, and no code is NaN */
#define PCD_KV_INT8 2 /* signed integers, -127 .. 127 */
typedef struct {
  void *k, *v;
  float *k_scale, *v_scale;
  int64_t page_stride, head_stride, token_stride;
  int n_pages, page_size, n_kv_heads, head_dim, format;
} pcd_kv_pages;

/* Both calls below take ragged sequences: rows q_off[s] .. q_off[s + 1) of
 * the n_tok rows belong to sequence s (n_seq + 1 non-decreasing offsets; a
 * sequence may have none, and rows behind the last offset are left alone),
 * kv_len[s] counts the sequence's tokens in the cache with the new ones
 * included, and token j of it lies in page table[s * table_stride + j /
 * page_size], slot j % page_size.  A row of the table has table_stride entries;
 * the forms ending in _cols take tables whose rows are the first table_width
 * entries (at most table_stride) of wider ones, as a column slice has them: a
 * length beyond those is out of range, and nothing behind them is read.
 * Offsets that decrease or leave the rows are reported, and the rows of their
 * sequences are left alone; work finds its sequence by a search, so rows of other
 * sequences of such a call may be left alone too.
 *
 * Append: the n new tokens of sequence s become its tokens kv_len[s] - n ..
 * kv_len[s] - 1.  k, v [n_tok][n_kv_heads][head_dim] of `dtype` (strides in
 * elements, channels contiguous).  Keys are rotated first, as by pcd_k_rope,
 * at pos[row] or, when pos is NULL, at their place in the sequence; freqs NULL
 * with rot_dim 0 stores them as they are.  A page's scale is set by its new
 * rows' largest |x|: over 448 rounded up to a power of two (e4m3) or over 127
 * (int8), at least 2^-60; while older tokens of the sequence stay in the
 * page it only grows, and their codes are then rescaled (e4m3: by a power of
 * two, exact while they stay normal; int8: rounded once more).  Codes round to
 * nearest even.  A NaN or infinity in a block's rows makes its scale so, and
 * all that is read from that block NaN.  A page that one call appends to
 * belongs to one sequence and stands once in its row of the table.  Nothing but the new tokens' pages is written.
 * Strides that put two rows of the cache in one place are refused, and keys and
 * values in one place. */
int pcd_k_kv_append(const pcd_kv_pages* cache, const void* k, const void* v, int dtype, int64_t k_tok, int64_t k_head,
                    int64_t v_tok, int64_t v_head, const int32_t* q_off, const int32_t* kv_len, const int32_t* table,
                    int n_seq, int n_tok, int table_stride, const int64_t* freqs, int rot_dim, int interleaved,
                    float amp, const int32_t* pos, int* dev_err, void* stream);
int pcd_k_kv_append_cols(const pcd_kv_pages* cache, const void* k, const void* v, int dtype, int64_t k_tok,
                         int64_t k_head, int64_t v_tok, int64_t v_head, const int32_t* q_off, const int32_t* kv_len,
                         const int32_t* table, int n_seq, int n_tok, int table_stride, int table_width,
                         const int64_t* freqs, int rot_dim, int interleaved, float amp, const int32_t* pos, int* dev_err,
                         void* stream);

/* Attention of q [n_tok][n_q_heads][head_dim] (dtype PCD_DTYPE_F16 or _BF16)
 * over the cache: out = softmax(scale q k^T) v per query head, query head h
 * reading KV head h / (n_q_heads / n_kv_heads).  causal != 0: row i of the n of
 * sequence s is its token kv_len[s] - n + i and sees the tokens up to itself
 * (rows before the cache's first token see none); causal == 0: every row sees
 * all kv_len[s] tokens, as branch rows see their shared prefix (How TypeSafe's
 * Jev Might Work, "One forward pass for all fields").  `lse` (may be NULL)
 * [n_tok][n_q_heads] fp32 receives the natural log-sum-exp of the scaled
 * scores, to join the result with attention over other keys.  A row that sees
 * nothing gives zeros and -inf.  Scores, softmax sums and the output are
 * accumulated in fp32; codes enter the products exactly and a value's scale
 * joins the softmax weight before its rounding to fp16 (the value scales that a
 * row sees may lie 2^100 apart).  A cache that was not written here holds no NaN
 * code (e4m3 0x7f, 0xff): it would reach rows that do not see its token; a NaN or
 * infinite scale reaches only rows that do.  Keys of a page that the table has
 * out of range are not seen; a length beyond the table reads as zero tokens.
 * `out` may be q's own view; another overlap is refused, as are strides that put
 * two of its rows in one place.
 * max_kv: the longest kv_len, as far as the host knows it; it sets how many
 * key ranges run side by side, not what is computed.  `scratch`: 16-byte
 * aligned, at least pcd_k_paged_attention_scratch_bytes (the same sizes, the
 * same GPU) bytes that the call overwrites; calls that may overlap in time,
 * captured graphs among them, need their own. */
int64_t pcd_k_paged_attention_scratch_bytes(int n_tok, int n_seq, int n_q_heads, int n_kv_heads, int head_dim,
                                            int64_t max_kv);
int pcd_k_paged_attention(const pcd_kv_pages* cache, const void* q, void* out, float* lse, int dtype, int n_q_heads,
                          int64_t q_tok, int64_t q_head, int64_t out_tok, int64_t out_head, const int32_t* q_off,
                          const int32_t* kv_len, const int32_t* table, int n_seq, int n_tok, int table_stride,
                          int64_t max_kv, int causal, float scale, void* scratch, int64_t scratch_bytes, int* dev_err,
                          void* stream);
int pcd_k_paged_attention_cols(const pcd_kv_pages* cache, const void* q, void* out, float* lse, int dtype, int n_q_heads,
                               int64_t q_tok, int64_t q_head, int64_t out_tok, int64_t out_head, const int32_t* q_off,
                               const int32_t* kv_len, const int32_t* table, int n_seq, int n_tok, int table_stride,
                               int table_width, int64_t max_kv, int causal, float scale, void* scratch,
                               int64_t scratch_bytes, int* dev_err, void* stream);

#ifdef __cplusplus
}
#endif
#endif
