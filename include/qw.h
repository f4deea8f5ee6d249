/*
 * qw.h - C ABI of libqw, a GB300 (sm_103a) implementation of the forward pass of a
 * Qwen2-style decoder-only transformer: prompt prefill into a preallocated KV cache and
 * KV-cached greedy decode.
 *
 * The operations follow these pages (cited by title and section):
 *   [LSA] "LLM Speedrun: Architecture": Transformer architecture (attention, causal mask,
 *         SwiGLU FFN, pre-norm residual stacking, GQA, RoPE, Decoding / LM head / KV
 *         cache) and Implementing Qwen (q/k/v bias, split-half RoPE, the model code's
 *         Decoder.step and generate_tokens).
 *   [AUG] "augur": Features (prefill/decode split, preallocated KV cache, greedy
 *         generation, EOS stopping).
 *   [QIE] "Building a Qwen2.5-1.5B Inference Engine From Scratch": §1 (prefill is
 *         compute-bound, decode is memory-bandwidth-bound).
 *
 * Conventions for every call:
 *   - Every call returns a qw_status; nothing aborts and nothing throws across the ABI.
 *     qw_last_error() gives a message for the last failing call on the calling thread.
 *   - "device" pointers are CUDA global-memory addresses on the device that was current
 *     when qw_create ran; "host" pointers are ordinary CPU memory.
 *   - Weights are BORROWED: the caller owns them, keeps them alive and unchanged until
 *     qw_destroy, and the library never writes them.
 *   - The library OWNS the KV cache, activations, logits, the RoPE table and the CUDA
 *     graph of a decode step; all are released by qw_destroy.
 *   - Work runs on the stream given to qw_create (or a stream the library creates when
 *     that argument is NULL). Calls that return host values synchronise that stream
 *     before returning.
 *   - After QW_ERR_CUDA or QW_ERR_TIMEOUT the model must be destroyed.
 */
#ifndef QW_H
#define QW_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QW_OK = 0,
  QW_ERR_INVALID_ARG = 1,   /* null pointer, bad size, inconsistent config */
  QW_ERR_UNSUPPORTED = 2,   /* a shape the library has no kernel for */
  QW_ERR_CAPACITY = 3,      /* a sequence would exceed kv_capacity */
  QW_ERR_TOKEN_RANGE = 4,   /* a token id outside [0, vocab) */
  QW_ERR_CUDA = 5,          /* a CUDA runtime call failed; destroy the model */
  QW_ERR_TIMEOUT = 6,       /* a bounded device-side wait gave up; destroy the model */
  QW_ERR_FAULT_INJECTED = 7,/* QW_FAULT environment variable forced a failure */
  QW_ERR_NUMERIC = 8        /* non-finite logits, or a value outside the fp16 range of the
                               KV cache (QW_BF16 models) or of a tensor-core operand */
} qw_status;

typedef enum { QW_F32 = 0, QW_BF16 = 1, QW_F16 = 2 } qw_dtype;

/* Model shape [LSA Implementing Qwen, the model configuration; AUG Qwen model config].
 * head_dim must be even and equal hidden / n_heads (the score scale 1/sqrt(d_k) uses
 * d_k = hidden / n_heads); n_heads must be a multiple of n_kv_heads. dtype is the storage
 * type of the weights, QW_F32 or QW_BF16. The KV cache is fp32 for QW_F32 models and fp16
 * for QW_BF16 models (same two bytes as bf16, eight times finer rounding); decode
 * activations, accumulators and logits are fp32; the prefill projections of QW_BF16 models
 * run on the tensor cores with fp16 operands (fp16 copies of the weights made by qw_create:
 * exact for 2^-17 <= |w| <= 65504, smaller weights round to a multiple of 2^-24, larger ones
 * are rejected) and fp32 accumulation. A key, value or operand that would overflow fp16 is
 * reported as QW_ERR_NUMERIC by the next call that checks device errors. */
typedef struct {
  int32_t n_layers, hidden, n_heads, n_kv_heads, head_dim, intermediate, vocab;
  float rms_eps;          /* RMSNorm epsilon, inside the square root (1e-6) */
  float rope_theta;       /* RoPE base (1e6) */
  int32_t tied_embeddings;/* 1: LM head is the embedding matrix */
  int32_t qkv_bias;       /* 1: q/k/v projections carry a bias [LSA Introducing bias] */
  int32_t dtype;          /* qw_dtype */
  int32_t max_seqs;       /* independent sequences held at once (1..16) */
  int32_t kv_capacity;    /* positions per sequence in the preallocated KV cache */
} qw_config;

/* Device pointers of one decoder layer, row-major [out, in], in qw_config.dtype.
 * Sizes: in_norm, post_norm [hidden]; wq [n_heads*head_dim, hidden]; wk, wv
 * [n_kv_heads*head_dim, hidden]; bq/bk/bv the matching vectors (NULL when qkv_bias is 0);
 * wo [hidden, n_heads*head_dim]; w_gate, w_up [intermediate, hidden];
 * w_down [hidden, intermediate]. Every pointer must be 16-byte aligned. */
typedef struct {
  const void *in_norm, *wq, *bq, *wk, *bk, *wv, *bv, *wo, *post_norm, *w_gate, *w_up,
      *w_down;
} qw_layer_weights;

/* embed [vocab, hidden]; final_norm [hidden]; lm_head [vocab, hidden] or NULL when tied;
 * layers is a HOST array of n_layers entries (copied by qw_create). */
typedef struct {
  const void *embed, *final_norm, *lm_head;
  const qw_layer_weights *layers;
} qw_weights;

typedef struct qw_model qw_model;

/* Build a model from its configuration and borrowed weights [LSA Implementing Qwen: the
 * model configuration and the Decoder that holds the embedding, the layers, the final
 * norm and the LM head; AUG Features: preallocated KV cache]. Validates the shape,
 * allocates the KV cache [max_seqs][n_layers][2][n_kv_heads][kv_capacity][head_dim] and
 * the working buffers, and builds the RoPE cos/sin table [LSA RoPE: angle = position *
 * theta^(-2i/head_dim)] with float64 angles on the host. cuda_stream is a cudaStream_t or
 * NULL. On success *out holds the model (release it with qw_destroy); on failure *out is
 * NULL and nothing stays allocated. Errors: QW_ERR_INVALID_ARG for a null, misaligned or
 * inconsistent argument, QW_ERR_UNSUPPORTED for a shape without kernels, QW_ERR_CUDA when
 * no GPU is usable or an allocation fails, QW_ERR_FAULT_INJECTED under QW_FAULT=alloc. */
qw_status qw_create(const qw_config *cfg, const qw_weights *w, void *cuda_stream,
                    qw_model **out);
void qw_destroy(qw_model *m);

/* Prefill [AUG Prefill/decode split; LSA Decoder.step on the whole prompt]: reset
 * sequence `seq`, run the n prompt tokens (host array) at positions 0..n-1, fill their
 * keys and values into the cache and compute the logits of the last position and its
 * greedy token. Afterwards the sequence holds n positions and its next decode step feeds
 * that token. next_token (host, may be NULL) receives it. Errors: QW_ERR_CAPACITY when
 * n > kv_capacity, QW_ERR_TOKEN_RANGE for an id outside [0, vocab). */
qw_status qw_prefill(qw_model *m, int32_t seq, const int32_t *ids, int32_t n,
                     int32_t *next_token);

/* The same with the prompt already in device memory; nothing is copied back and the
 * stream is not synchronised (token ids are range-checked on the device, reported by
 * qw_sync). */
qw_status qw_prefill_device(qw_model *m, int32_t seq, const int32_t *ids_dev, int32_t n);

/* One greedy decode step [LSA Decoding / KV cache; AUG greedy generation] for every
 * sequence that has been prefilled: run one token at position pos (the sequence's current
 * length), append its key and value at pos, compute the logits and the argmax, and
 * advance the length by one. feed (host [max_seqs], may be NULL) overrides the token run
 * for each sequence (teacher forcing); NULL runs each sequence's previous greedy token.
 * next_tokens (host [max_seqs], may be NULL) receives the new tokens; when it is NULL the
 * call does not synchronise. Errors: QW_ERR_CAPACITY when a sequence is full. */
qw_status qw_decode_step(qw_model *m, const int32_t *feed, int32_t *next_tokens);

/* n_steps decode steps of every active sequence, each feeding its own greedy token, with
 * no host synchronisation. Tokens are kept on the device (qw_tokens_device). */
qw_status qw_decode_steps(qw_model *m, int32_t n_steps);

/* Greedy generation of one sequence (seq 0) [AUG EOS stopping; LSA generate_tokens]:
 * prefill the n prompt ids (host), then decode until max_new tokens exist in total (the
 * prefill's token counts) or a token equal to eos (eos < 0: never) has been produced; that
 * token is kept. out (host [max_new]) receives the tokens, n_out their number. */
qw_status qw_generate(qw_model *m, const int32_t *ids, int32_t n, int32_t max_new,
                      int32_t eos, int32_t *out, int32_t *n_out);

/* The same with a set of stop ids [LSA Implementing Qwen: generate_tokens stops on any id of
 * its eos_ids set, the chat template's end tokens among them]: generation stops after the
 * first produced token that equals any of stop_ids[0 .. n_stop-1] (host array, may hold
 * duplicates; n_stop = 0: no stop id). That token is kept, and the sequence continues
 * from it as after qw_generate. Errors: QW_ERR_INVALID_ARG for n_stop < 0 or a null
 * stop_ids with n_stop > 0, and those of qw_generate. */
qw_status qw_generate_stops(qw_model *m, const int32_t *ids, int32_t n, int32_t max_new,
                            const int32_t *stop_ids, int32_t n_stop, int32_t *out,
                            int32_t *n_out);

/* Wait for queued work and report a device-side error (token range, non-finite logits). */
qw_status qw_sync(qw_model *m);

/* Device pointer to the fp32 logits [max_seqs][vocab] of the last step [LSA Decoding and
 * Decoder.step: the logits of the last position, LM head applied to the final norm];
 * row seq holds sequence seq's. Owned by the model; valid until the next call that runs
 * it. NULL for a null model. */
const float *qw_logits(const qw_model *m);

/* Copy the fp32 logits [vocab] of sequence seq's last step to host memory (synchronises). */
qw_status qw_read_logits(qw_model *m, int32_t seq, float *host_out);

/* Device pointer to int32 [max_seqs]: the greedy token of each sequence's last step. */
const int32_t *qw_tokens_device(const qw_model *m);

/* Current length of sequence seq: the positions its KV cache holds, which is also the
 * position the next decode step runs at [LSA Decoder.step: positions of the new token;
 * KV cache]. 0 for a sequence that is not active. Errors: QW_ERR_INVALID_ARG. */
qw_status qw_position(const qw_model *m, int32_t seq, int32_t *pos);

/* Kernel launches one single-sequence decode step makes: 1 when the step runs as one
 * persistent kernel (bf16 models whose shape it supports, the default), else
 * n_layers * 5 + 2 (embedding, q/k/v, attention, o_proj, gate/up, down per layer, LM head).
 * 0 for a null model. */
int32_t qw_decode_kernels_per_step(const qw_model *m);

/* Forget sequence seq [LSA KVCache: a fresh cache per sequence; AUG Features:
 * preallocated KV cache]: its length becomes 0 and it leaves the set of active sequences;
 * its cache rows are overwritten by its next prefill. Does not synchronise. Errors:
 * QW_ERR_INVALID_ARG for a null model or a sequence index outside [0, max_seqs). */
qw_status qw_reset(qw_model *m, int32_t seq);

/* Profiling hook. With begin and end non-NULL (host arrays of n_layers cudaEvent_t created
 * with timing enabled), every later decode step records begin[l] just before and end[l]
 * just after kernel `kind` of layer l: 0 qkv, 1 attention, 2 o_proj, 3 gate/up, 4 down;
 * kind 5 is the LM head (begin[0], end[0] only). The traced kernel and the one after it
 * then launch without programmatic dependent launch. NULL arrays remove the hook. The
 * decode graphs are rebuilt on the next step. */
qw_status qw_set_trace(qw_model *m, int32_t kind, void *const *begin, void *const *end);

/* Device timeline (profiling). With enable 1, every later decode step records, for each of
 * its kernel launches (embedding, then per layer qkv, attention, o_proj, gate/up, down, then
 * the LM head), three %globaltimer stamps in ns: the first CTA's start, the first CTA past
 * its wait for the previous kernel, and the last CTA's end. qw_read_timeline copies the
 * stamps of the last step, 3 per launch in launch order, into out (host, 3 * max_launches
 * uint64) and the launch count into n_launches. Timing differs slightly from an
 * uninstrumented run (one atomic per CTA per stamp). enable 0 frees the buffer.
 * When a single-sequence step runs as one persistent kernel (qw_decode_kernels_per_step
 * is 1), entry k < 5 * n_layers + 1 is phase k of the step instead (q/k/v, attention,
 * o_proj, gate/up, down per layer, then the LM head): [start after the previous grid
 * barrier, its weight units consumed, end before the next grid barrier], stamped by the
 * first CTA. */
qw_status qw_set_timeline(qw_model *m, int32_t enable);
qw_status qw_read_timeline(qw_model *m, uint64_t *out, int32_t max_launches, int32_t *n_launches);

/* Message for the last failing call on this thread ("" if none). */
const char *qw_last_error(void);

/* ---- single operations, for testing a step of the path in isolation ---- */

/* GQA decode attention of one token [LSA Attention, Causal mask, GQA]: for every query
 * head h, scores s_j = q_h . K_j / sqrt(head_dim) over positions j = 0..ctx-1 of KV head
 * h / (n_heads / n_kv_heads), softmax, and out_h = sum_j p_j V_j. The context is split
 * into chunks whose partial softmax statistics are merged exactly (log-sum-exp).
 *   q    device fp32 [n_heads*head_dim]
 *   k, v device, kv_dtype (QW_F32 or QW_F16) elements, [n_kv_heads][kv_stride][head_dim]
 *        (position-major per head), ctx <= kv_stride
 *   out  device fp32 [n_heads*head_dim]
 *   workspace device, at least qw_op_decode_attention_workspace() bytes, 16-byte
 *        aligned; its counters must be zero before the first call (cudaMemset) and the
 *        call leaves them zero again.
 * Shapes: head_dim a multiple of 8, at most 8 query heads per KV head and
 * (n_heads / n_kv_heads) * head_dim <= 1024; others return QW_ERR_UNSUPPORTED.
 * Runs on cuda_stream (NULL = default stream) and does not synchronise. */
size_t qw_op_decode_attention_workspace(int32_t n_heads, int32_t n_kv_heads,
                                        int32_t head_dim, int32_t max_ctx);
qw_status qw_op_decode_attention(int32_t kv_dtype, int32_t n_heads, int32_t n_kv_heads,
                                 int32_t head_dim, int32_t ctx, int32_t kv_stride,
                                 const float *q, const void *k, const void *v, float *out,
                                 void *workspace, size_t workspace_bytes,
                                 void *cuda_stream);

/* Decode attention for callers that cannot allocate device memory. The pages have no
 * counterpart: this is a deployment variant of qw_op_decode_attention, computing the same
 * result (same kernel) with its scratch (the split-context partials and the per-KV-head
 * counters) in one fixed 1 MiB array inside the library instead of a caller workspace.
 * It is meant for callers that cannot call cudaMalloc where they call attention: code
 * embedded in another runtime that owns all device memory, or loops that must not pay
 * cudaMalloc's implicit device synchronisation or risk an allocation failure mid-run.
 *   - Arguments, layouts and errors are those of qw_op_decode_attention, without the
 *     workspace. Shapes whose scratch exceeds qw_op_decode_attention_noalloc_limit()
 *     bytes are rejected with QW_ERR_UNSUPPORTED (1 MiB fits, for example, 12 query /
 *     2 KV heads of dimension 128 with kv_stride up to 8192).
 *   - Nothing is allocated: no cudaMalloc, cudaFree or allocating library routine. Every
 *     GPU that loads the library holds the array until the process exits.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress,
 *     with that device current); make that first call before any stream capture. A first
 *     call on a stream that is capturing returns QW_ERR_INVALID_ARG and does nothing.
 *   - Each call clears the counters it needs (cudaMemsetAsync on cuda_stream). All calls
 *     share the one array: calls that overlap on the GPU (other streams, other threads)
 *     race on it and must be serialised by the caller. */
qw_status qw_op_decode_attention_noalloc(int32_t kv_dtype, int32_t n_heads, int32_t n_kv_heads,
                                         int32_t head_dim, int32_t ctx, int32_t kv_stride,
                                         const float *q, const void *k, const void *v,
                                         float *out, void *cuda_stream);
size_t qw_op_decode_attention_noalloc_limit(void);

/* Dense GEMM on the tensor cores (tcgen05), the contraction of every prefill projection
 * [LSA Implementing Qwen: W @ x for all prompt columns at once; QIE §1: prefill is
 * compute-bound]: C[M][N] = A[M][K] . B[N][K]^T (+ bias[N]), or C += A . B^T when
 * accumulate is 1 (the residual add). A, B fp16 row-major, bias bf16 (may be NULL), C fp32
 * row-major, all device, contiguous (row pitch = K for A and B, N for C), 16-byte aligned;
 * K and N multiples of 8. err_dev is a device int32 that receives QW device error bits (a
 * bounded wait that expired). Runs on cuda_stream without synchronising. */
qw_status qw_op_gemm_f16(int32_t M, int32_t N, int32_t K, const void *A, const void *B,
                          const void *bias, float *C, int32_t accumulate, int32_t *err_dev,
                          void *cuda_stream);

/* Fused gate/up projection and SwiGLU [LSA SwiGLU FFN]: act[M][N] =
 * silu(A . Wg^T) * (A . Wu^T), A [M][K], Wg/Wu [N][K] fp16, act fp16 [M][N]; the same
 * layout rules as qw_op_gemm_f16. */
qw_status qw_op_gemm_swiglu_f16(int32_t M, int32_t N, int32_t K, const void *A,
                                 const void *Wg, const void *Wu, void *act, int32_t *err_dev,
                                 void *cuda_stream);

/* ---- a paged key-value cache and the operators around it ----
 *
 * One serving step of many sequences: qw_op_page_plan hands out pages and says where each new
 * token goes, qw_op_rope_append rotates the queries and keys and writes keys and values
 * there, qw_op_paged_attention reads the pages back for one new token per sequence, and
 * qw_op_token_logprobs turns the step's logits into log probabilities.
 * qw_op_page_release returns the pages of finished sequences. Where several sequences go on from one prompt (samples, beams),
 * qw_op_page_fork lets them share its pages, qw_op_shared_attention reads them once, qw_op_beam_select chooses how the beams go
 * on, and qw_op_page_copy and qw_op_page_compact move pages.
 *
 * Conventions of these calls:
 *   - All pointers are device pointers on the current device unless marked host; a pointer to
 *     host memory or to another device's is refused (QW_ERR_INVALID_ARG), and so is one that is
 *     not aligned to its elements. The stream belongs to the current device. Nothing is allocated
 *     and nothing synchronises; every call may be captured into a CUDA graph, which then reads
 *     the lengths, tables and counts that the device memory holds at each replay.
 *   - What only the device can see (lengths, page ids, slots, token ids) is checked there:
 *     a bad value is never used as an address, and its QW_DEV_* bit is OR-ed into err_dev
 *     (device int32, required, never cleared by the library).
 *   - Zero sequences, tokens or rows are allowed and do nothing, unless stated otherwise.
 *   - Tensors of one call must not overlap, unless stated otherwise. */

/* Bits of a device error word (err_dev). */
enum {
  QW_DEV_TOKEN = 1,      /* a token id outside [0, vocab) */
  QW_DEV_NONFINITE = 2,  /* a row of logits without a distribution */
  QW_DEV_TIMEOUT = 4,    /* a bounded wait gave up */
  QW_DEV_RANGE = 8,      /* a value outside the fp16 range (stored as an infinity), or not finite */
  QW_DEV_LAYOUT = 16,    /* shared memory found misaligned; the work was skipped */
  QW_DEV_PAGE = 32,      /* a page id, slot or length outside the cache */
  QW_DEV_CAPACITY = 64   /* a page plan that does not fit; nothing was handed out */
};

/* One layer's cache: n_pages pages of page_size positions. Element (page p, KV head h, position
 * i of the page, dimension d) of the keys lies at k[p * page_stride + h * head_stride +
 * i * pos_stride + d], of the values at the same place of v; strides are in elements of dtype
 * (QW_F32, QW_F16 or QW_BF16). Either [page][head][position] or [page][position][head] order,
 * with gaps allowed between rows, heads and pages; a stride along an extent of 1 is not
 * looked at. k and v are 16-byte aligned, the strides multiples of 16 bytes. head_dim is a
 * multiple of 8, at most 256. Slot s of the cache is position s % page_size of page
 * s / page_size. The struct itself is host memory and is read during the call only. */
typedef struct {
  void *k, *v;
  int32_t dtype, n_pages, page_size, n_kv_heads, head_dim;
  int64_t page_stride, head_stride, pos_stride;
} qw_paged_kv;

/* Page plan of one step: takes pages for the new tokens of every sequence from a list of free
 * pages and says where each token goes. Sequence b holds lens[b] positions in the pages
 * block_table[b][0 .. ceil(lens[b] / page_size) - 1] and gets n_new[b] >= 0 more (n_new NULL: one
 * each). Its further pages are taken from the end of free_pages[0 .. n_free[0] - 1]: the i-th page
 * taken, counted over sequences in order and over a sequence's pages in order, is
 * free_pages[n_free[0] - 1 - i].
 *   block_table  [n_seqs][max_blocks], in and out: the new pages' entries are written
 *   lens_out     [n_seqs]: lens + n_new; may be lens
 *   n_free_out   [1]: what is left of free_pages, which is not written; may be n_free
 *   cu_tokens    [n_seqs + 1]: token t of the step belongs to the sequence b with
 *                cu_tokens[b] <= t < cu_tokens[b + 1]
 *   positions    [max_tokens]: lens[b] + t - cu_tokens[b]; 0 behind the last token
 *   slots        [max_tokens]: the token's slot in the cache; -1 behind the last token
 * If the step does not fit (too few free pages, more than max_tokens tokens, more than max_blocks
 * pages or 2^31 - 1 positions of a sequence, a negative length or count, n_free outside
 * [0, n_pages]) QW_DEV_CAPACITY is set and the step is empty: lens_out = lens, n_free_out = n_free, cu_tokens 0, positions 0,
 * slots -1. A page id outside [0, n_pages) gives slot -1 and sets QW_DEV_PAGE. n_seqs <= 16384,
 * n_pages and max_tokens <= 2^30.
 * With n_seqs = 0 the outputs are those of an empty step. max_tokens = 0 is allowed. */
qw_status qw_op_page_plan(int32_t n_seqs, int32_t page_size, int32_t n_pages, int32_t max_blocks, int32_t max_tokens,
                          const int32_t *lens, const int32_t *n_new, const int32_t *free_pages,
                          const int32_t *n_free, int32_t *block_table, int32_t *lens_out,
                          int32_t *n_free_out, int32_t *cu_tokens, int32_t *positions, int64_t *slots,
                          int32_t *err_dev, void *cuda_stream);

/* Gives the pages of finished sequences back: for every b with done[b] != 0, in order, its pages
 * block_table[b][0 .. ceil(lens[b] / page_size) - 1] are appended to free_pages (device
 * [n_pages]) behind its first n_free[0] entries. lens_out[b] is 0 for those sequences and
 * lens[b] for the others (lens_out may be lens); n_free_out is the new count (may be n_free).
 * The table is not written. If the list would exceed n_pages, a length is negative or beyond
 * max_blocks pages, or n_free is outside [0, n_pages], QW_DEV_CAPACITY is set, lens_out = lens
 * and n_free_out = n_free, and no page moves. A page id outside [0, n_pages) moves as it is and
 * sets QW_DEV_PAGE. n_seqs <= 16384, n_pages <= 2^30. */
qw_status qw_op_page_release(int32_t n_seqs, int32_t page_size, int32_t n_pages, int32_t max_blocks,
                             const int32_t *lens, const int32_t *done, const int32_t *block_table,
                             int32_t *free_pages, const int32_t *n_free, int32_t *lens_out,
                             int32_t *n_free_out, int32_t *err_dev, void *cuda_stream);

/* Forks sequences, and ends those that nobody goes on from: sequence i of the n_out new ones is a copy of the old
 * sequence parents[i] (-1: an empty one) that shares its pages. shares[p] is the number of holders of page p (rows of
 * block tables) beyond the first: 0 for pages of one holder and for free ones, so that pages from qw_op_page_plan need no
 * entry. A last page that is partly filled is written by the next append, so only the lowest child of its parent keeps
 * it; every other child, in order, takes a page from the end of free_pages[0 .. n_free[0] - 1] for it:
 *   lens_out [n_out], table_out [n_out][max_blocks]: the new sequences; entries behind a sequence's pages are not written
 *   copy_src, copy_dst, copy_len [n_out]: that child's old and new last page and its positions, for qw_op_page_copy; -1, -1
 *       and 0 where nothing is to be copied
 *   shares_out [n_pages]; may be shares
 *   free_out [n_pages]: the free pages that were not taken, in their order, then the pages whose last holder ended, in
 *       ascending order; may be free_pages. n_free_out [1] their number; may be n_free
 * A sequence ends where no child names it: with parents[i] = i or -1 the call returns the pages of finished sequences to
 * the list (qw_op_page_release does so for pages that nobody shares). Of the pages in parents' tables shares counts
 * other holders too, such as a kept prompt's. lens_out and table_out must be other memory than lens and block_table.
 * If there are too few free pages, a length is negative or beyond max_blocks pages, or n_free is outside [0, n_pages],
 * QW_DEV_CAPACITY is set and nothing is forked, ended or taken: lens_out 0, nothing to copy, shares, list and count as they
 * were. A parent outside [-1, n_seqs) counts as -1, a page id outside [0, n_pages) is copied and not counted, and a list that would
 * have more than n_pages pages (some were held and on it) ends there; all three set QW_DEV_PAGE. A negative count is taken as 0.
 * A partly filled last page has no other holder than its row (every fork leaves it so): the child that keeps it appends to it.
 * n_seqs and n_out <= 16384, n_pages <= 2^30.
 * workspace: at least qw_op_page_fork_workspace() bytes, 16-byte aligned, zeroed once before its first use; it serves this
 * call alone, and every call leaves it ready for the next with the same n_pages. Calls that may run at the same time need
 * workspaces of their own. */
size_t qw_op_page_fork_workspace(int32_t n_pages);
qw_status qw_op_page_fork(int32_t n_seqs, int32_t n_out, int32_t page_size, int32_t n_pages, int32_t max_blocks,
                          const int32_t *lens, const int32_t *block_table, const int32_t *parents, const int32_t *shares,
                          const int32_t *free_pages, const int32_t *n_free, int32_t *lens_out, int32_t *table_out,
                          int32_t *shares_out, int32_t *free_out, int32_t *n_free_out, int32_t *copy_src,
                          int32_t *copy_dst, int32_t *copy_len, void *workspace, size_t workspace_bytes,
                          int32_t *err_dev, void *cuda_stream);

/* Compacts the pool: pages that are not among free_pages[0 .. n_free[0] - 1] are live, L of them. The i-th highest live
 * page of an id >= L moves to the i-th lowest free page of an id < L, i < n_moves[0] = min(their number, max_moves):
 *   move_src, move_dst [max_moves]: the moves, -1 behind the last. qw_op_page_copy carries them out (in every cache of
 *       the pool, before anything else reads it)
 *   table_out [n_seqs][max_blocks]: the tables with the moved pages' new ids; may be block_table
 *   shares_out [n_pages]: the pages' counts (see qw_op_page_fork) carried along; may be shares. Both NULL: no page is shared
 *   free_out [n_pages]: the free pages afterwards in descending order, so that the lowest are taken first; may be free_pages.
 *       Their number stays n_free[0]
 * Other tables of the same pool can be rewritten from the moves. If a page is on the list twice or outside
 * [0, n_pages) (QW_DEV_PAGE), or n_free or a length is out of range (QW_DEV_CAPACITY), nothing moves and the outputs are
 * the inputs. Else a table entry outside [0, n_pages) stays and sets QW_DEV_PAGE, whether pages move or not. n_pages and
 * max_moves <= 2^30.
 * workspace: at least qw_op_page_compact_workspace() bytes, with the rules of qw_op_page_fork's. */
size_t qw_op_page_compact_workspace(int32_t n_pages);
qw_status qw_op_page_compact(int32_t n_seqs, int32_t page_size, int32_t n_pages, int32_t max_blocks, int32_t max_moves,
                             const int32_t *lens, const int32_t *block_table, const int32_t *shares,
                             const int32_t *free_pages, const int32_t *n_free, int32_t *table_out, int32_t *shares_out,
                             int32_t *free_out, int32_t *move_src, int32_t *move_dst, int32_t *n_moves, void *workspace,
                             size_t workspace_bytes, int32_t *err_dev, void *cuda_stream);

/* Copies pages inside n_caches caches (host array; the layers of one model, which have the same type, extents and
 * strides; at most 128): for every i < n with src[i] != -1 the first len[i] positions (len NULL: all) of page src[i], in all
 * heads, keys and values, to page dst[i]. No two entries have the same dst, and no dst is a src. A page outside
 * [0, n_pages), or a length outside [0, page_size], copies nothing and sets QW_DEV_PAGE. */
qw_status qw_op_page_copy(const qw_paged_kv *caches, int32_t n_caches, int32_t n, const int32_t *src, const int32_t *dst,
                          const int32_t *len, int32_t *err_dev, void *cuda_stream);

/* How rotary frequencies are stretched for contexts longer than the trained one. With r the
 * rotated dimensions, w_i = theta^(-2i/r), i < r/2, and L = orig_len:
 *   QW_ROPE_NONE    w_i
 *   QW_ROPE_LINEAR  w_i / factor
 *   QW_ROPE_NTK     theta replaced by theta * factor^(r / (r - 2))
 *   QW_ROPE_YARN    (1 - c_i) w_i + c_i w_i / factor, c_i rising linearly from 0 to 1 between
 *                   the indices (rounded outwards, inside [0, r - 1]) whose frequency turns
 *                   `high` and `low` times over L positions; cos and sin times
 *                   0.1 ln(factor) + 1
 *   QW_ROPE_BANDS   w_i / factor where L w_i / 2 pi <= low, w_i where it is >= high, and a
 *                   linear blend in L w_i / 2 pi between them */
typedef enum { QW_ROPE_NONE = 0, QW_ROPE_LINEAR = 1, QW_ROPE_NTK = 2, QW_ROPE_YARN = 3, QW_ROPE_BANDS = 4 } qw_rope_scaling;

/* The rotary frequencies of qw_op_rope_append, on the host (no GPU needed): turns[i] (host
 * [rot_dim / 2]) is w_i / 2 pi as a fraction of a turn in units of 2^-64, rounded; *mscale (host)
 * the factor of cos and sin. rot_dim even and positive, theta > 1, factor >= 1, orig_len > 0 and
 * 0 < low < high where the scaling uses them; else QW_ERR_INVALID_ARG. The fraction of a turn at
 * position p is then the low 64 bits of p * turns[i]: exact for every position. */
qw_status qw_rope_turns(int32_t rot_dim, double theta, int32_t scaling, double factor, double orig_len, double low,
                        double high, uint64_t *turns, float *mscale);

/* Rotary positions of the queries and keys of n_tokens tokens, and the append of the keys and
 * values to a paged cache [LSA RoPE; KV cache]. Token t stands at positions[t] (any int32). The
 * first rot_dim dimensions of every query and key head are rotated in pairs (a, b), pair i by
 * the angle positions[t] * w_i: a' = mscale (a cos - b sin), b' = mscale (a sin + b cos); the
 * pair is dimensions (i, i + rot_dim / 2), or (2i, 2i + 1) when adjacent is 1. The remaining
 * dimensions pass unchanged. q_out receives the queries, slot slots[t] of the cache the
 * rotated key and the value; slot -1 writes no key and value, a slot outside
 * [0, n_pages * page_size) neither, and sets QW_DEV_PAGE. Two tokens of a call must not have
 * the same slot (either's values may end up there).
 *   q [n_tokens][n_heads][head_dim], k, v [n_tokens][n_kv_heads][head_dim], all of io_dtype, heads
 *   contiguous, one token's row q_stride (k_stride, v_stride) elements after the last one's;
 *   q_out like q with q_out_stride. q_out may be q (with the same stride). All 16-byte aligned,
 *   strides multiples of 16 bytes; q, k and v may lie in one fused row.
 *   turns (device [rot_dim / 2]) and mscale as from qw_rope_turns; rot_dim even, 2 .. head_dim.
 * io_dtype QW_F32 with any cache type, or the cache's own type. Angles are reduced in 64-bit
 * fixed point, all else is fp32, rounded once. An fp16 result out of range, or not finite,
 * sets QW_DEV_RANGE. */
qw_status qw_op_rope_append(const qw_paged_kv *cache, int32_t n_tokens, int32_t n_heads, int32_t io_dtype,
                            const int32_t *positions, const int64_t *slots, const uint64_t *turns, int32_t rot_dim,
                            int32_t adjacent, float mscale, const void *q, int64_t q_stride, const void *k,
                            int64_t k_stride, const void *v, int64_t v_stride, void *q_out, int64_t q_out_stride,
                            int32_t *err_dev, void *cuda_stream);

/* GQA decode attention over a paged cache, one query token per sequence [LSA Attention, GQA]: for
 * sequence b and query head h, scores s_j = scale * q_h . K_j over the positions j = 0 ..
 * lens[b] - 1 of KV head h / (n_heads / n_kv_heads), out_h = sum_j softmax(s)_j V_j and
 * lse_h = ln sum_j exp(s_j). Position j lies in page block_table[b][j / page_size]; what the last
 * page holds behind it is not read. A sequence of length 0 gives out 0 and lse -inf.
 * A NaN among the keys, values or queries makes every output that it reaches NaN, an infinity
 * makes it infinite or NaN; other heads and sequences are not touched. A length that is negative or
 * beyond max_blocks pages is cut to that range, the positions of a page outside [0, n_pages)
 * are left out (out 0 and lse -inf if none remains), and both set QW_DEV_PAGE.
 *   block_table [n_seqs][max_blocks], max_blocks * page_size at most 2^30; lens [n_seqs]
 *   q   [n_seqs][n_heads][head_dim] of io_dtype, heads contiguous, q_stride elements between
 *       sequences; out the same with out_stride; both 16-byte aligned, strides multiples of
 *       16 bytes. out may be q (with the same stride).
 *   scale of a magnitude of at most 2^127
 *   lse fp32 [n_seqs][n_heads], or NULL
 *   workspace at least qw_op_paged_attention_workspace() bytes, 16-byte aligned, zeroed once
 *       before its first use (cudaMemset); every call leaves it ready for the next, of any
 *       shape and also of qw_op_token_logprobs. Calls that may run at the same time, captured
 *       graphs of them included, need workspaces of their own.
 * io_dtype QW_F32 with any cache type, or the cache's own type; sums are fp32 and divided at the
 * end, so values whose sum over the positions passes 2^118 overflow to infinities. Over an fp16
 * cache an fp32 query keeps 22 bits, of its head's largest element. Any n_heads that is
 * a multiple of the cache's n_kv_heads. The result does not depend on the run: equal inputs give
 * equal bits on equal devices. */
size_t qw_op_paged_attention_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim);
qw_status qw_op_paged_attention(const qw_paged_kv *cache, int32_t n_seqs, int32_t n_heads, const int32_t *block_table,
                                int32_t max_blocks, const int32_t *lens, int32_t io_dtype, const void *q,
                                int64_t q_stride, float scale, void *out, int64_t out_stride, float *lse,
                                void *workspace, size_t workspace_bytes, int32_t *err_dev, void *cuda_stream);

/* The same for groups of sequences that begin alike (samples or beams of one prompt, users of one system prompt): what is
 * shared is read once for the group. Group g is the sequences cu_seqs[g] .. cu_seqs[g + 1] - 1 (cu_seqs[0] = 0,
 * cu_seqs[n_groups] = n_seqs, some may be empty), and each of them shares its first shared_lens[b] positions with the
 * group's first sequence, whose table says where they lie (whatever its own length is): out and lse are those of
 * qw_op_paged_attention where every table holds these positions. shared_lens is one number in a group, or 0 for sequences
 * that share nothing; a sequence shorter than that is computed from its own table alone.
 * A sequence that claims to share another number of positions than the group's first sets QW_DEV_PAGE and misses them.
 * Bounds of groups that do not ascend from 0 to n_seqs set QW_DEV_PAGE, and all outputs are 0, lse -inf.
 *   cu_seqs [n_groups + 1], 1 <= n_groups <= n_seqs; shared_lens [n_seqs]
 *   workspace at least qw_op_shared_attention_workspace() bytes, with the rules of qw_op_paged_attention's, which it
 *       serves too
 * Probabilities keep two pieces of the cache's type (22 bits, bf16 16) for 16-bit callers and 22 bits and more for fp32 ones, as
 * there. A 16-bit caller's values whose sum over the shared positions passes 2^113 overflow. Equal inputs give equal bits on equal
 * devices.
 * It pays where it saves much: it takes three launches and sums partial results up, 7 to 30 us that qw_op_paged_attention does
 * not take. Where the groups' later sequences would read less than about 100 MB of shared keys and values in all, that call is faster,
 * over tables that hold the shared pages (as forks leave them). */
size_t qw_op_shared_attention_workspace(int32_t n_seqs, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim);
qw_status qw_op_shared_attention(const qw_paged_kv *cache, int32_t n_seqs, int32_t n_heads, const int32_t *block_table,
                                 int32_t max_blocks, const int32_t *lens, int32_t n_groups, const int32_t *cu_seqs,
                                 const int32_t *shared_lens, int32_t io_dtype, const void *q, int64_t q_stride, float scale,
                                 void *out, int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes,
                                 int32_t *err_dev, void *cuda_stream);

/* Log probabilities of given tokens, with their ranks, the entropy and the likeliest tokens, of
 * n_rows rows of logits [LSA Decoding: softmax of the logits]. For a row z:
 *   logprobs[i] = z_t - ln sum_j exp(z_j) for t = ids[i], i < n_ids
 *   ranks[i]    = 1 + the tokens with a larger logit, or the same and a lower id
 *   entropy     = - sum_j p_j ln p_j in nats (p = softmax(z); 0 where p_j is 0)
 *   top_ids, top_logprobs: the top_k tokens in that order, and their log probabilities
 * A logit of -inf is a token of probability 0; a log probability beyond fp32 is -inf. A row that
 * holds a NaN or +inf, or nothing but -inf, has no distribution: QW_DEV_NONFINITE is set, logprobs,
 * entropy and top_logprobs are NaN, ranks 0 and top_ids -1. An id of -1 marks no token (logprob 0,
 * rank 0); any other id outside [0, vocab) gives NaN and rank 0 and sets QW_DEV_TOKEN.
 *   logits [n_rows][row_stride >= vocab] of logits_dtype, aligned to its own size
 *   ids, logprobs, ranks [n_rows][n_ids], n_ids 0 .. 8 (0: all three may be NULL); ranks may be NULL
 *   entropy [n_rows] or NULL
 *   top_ids, top_logprobs [n_rows][top_k], top_k 0 .. min(32, vocab) (0: both may be NULL)
 *   workspace at least qw_op_token_logprobs_workspace() bytes, with the rules of
 *       qw_op_paged_attention's. Equal inputs give equal bits on equal devices. */
size_t qw_op_token_logprobs_workspace(int32_t n_rows, int32_t vocab, int32_t top_k);
qw_status qw_op_token_logprobs(int32_t logits_dtype, int32_t n_rows, int32_t vocab, const void *logits,
                               int64_t row_stride, const int32_t *ids, int32_t n_ids, float *logprobs, int32_t *ranks,
                               float *entropy, int32_t top_k, int32_t *top_ids, float *top_logprobs, void *workspace,
                               size_t workspace_bytes, int32_t *err_dev, void *cuda_stream);

/* A step of beam search for n_groups groups of n_beams beams [LSA Decoding: softmax of the logits]: row w = g * n_beams + i is
 * beam i of group g, scores[w] the sum of its tokens' log probabilities. The beam can go on with any token t of a logit
 * above -inf, and its score becomes scores[w] + z_t - ln sum_j exp(z_j); an ended beam (ended[w] != 0) stays as it is, a
 * single candidate with its own score and the token end_id. The n_out best of a group, by weights[w] * score, in order; equal
 * ones by the lower beam, then the larger logit, then the lower id. The order is that of the scores in 64 bits, whose
 * normaliser is exact to 1e-10 where tokens above 2^-10 carry a row (a beam with one token left keeps its score as it is),
 * to 2e-8 of wide rows, and to 2e-7 at worst (thousands of equal logits that carry a row together, logits beyond 2^20).
 *   logits [n_groups * n_beams][row_stride >= vocab] of logits_dtype, aligned to its own size
 *   scores [rows]; -inf: a beam that is not there. weights [rows], positive, such as a power of 1 / length; NULL: 1
 *   ended [rows] or NULL: none. end_id: the token that ends a beam, or -1
 *   parents, tokens, scores_out, ended_out [n_groups * n_out]: the candidate's row, token, score, and whether it has ended
 *       (its parent had, or its token is end_id); ended_out may be NULL. If there are fewer candidates than n_out, the rest
 *       is parent -1, token -1, score -inf, ended 1
 *   history, history_out [rows][width] and [n_groups * n_out][width], lens, lens_out [rows] and [n_groups * n_out]: the tokens of
 *       the beams so far in the order of the new beams, each with its token behind (an ended beam's stays), and their
 *       numbers; all NULL: none. What lies behind a history is not written. A history that is full, or a length outside
 *       [0, width], sets QW_DEV_CAPACITY; the history then stays as long as it is
 * A row whose logits hold a NaN or +inf, or nothing but -inf, whose score is NaN or +inf, or whose weight is not positive and
 * finite, has no candidates and sets QW_DEV_NONFINITE (the logits of ended and absent beams are not looked at).
 * The outputs are other memory than the inputs. parents can go to qw_op_page_fork as they are.
 * At most 65535 groups, 32 beams, 32 candidates, 2^21 tokens. workspace: at least qw_op_beam_select_workspace() bytes, 16-byte
 * aligned; it need not be zeroed. Calls that may run at the same time need workspaces of their own. Equal inputs
 * give equal bits on equal devices. */
size_t qw_op_beam_select_workspace(int32_t n_groups, int32_t n_beams, int32_t vocab, int32_t n_out);
qw_status qw_op_beam_select(int32_t logits_dtype, int32_t n_groups, int32_t n_beams, int32_t vocab, const void *logits,
                            int64_t row_stride, const float *scores, const float *weights, const int32_t *ended,
                            int32_t end_id, int32_t n_out, int32_t *parents, int32_t *tokens, float *scores_out,
                            int32_t *ended_out, int32_t width, const int32_t *history, const int32_t *lens,
                            int32_t *history_out, int32_t *lens_out, void *workspace, size_t workspace_bytes,
                            int32_t *err_dev, void *cuda_stream);

/* The same as qw_op_token_logprobs for the logits of sequence seq's last step, into host memory (all pointers host, sizes
 * and NULL rules as above, one row; entropy one float). The scratch is allocated by the first
 * call and released by qw_destroy. Synchronises. Errors: QW_ERR_INVALID_ARG for a sequence that
 * is not active, QW_ERR_TOKEN_RANGE for an id outside [0, vocab), QW_ERR_NUMERIC for
 * non-finite logits. */
qw_status qw_read_logprobs(qw_model *m, int32_t seq, const int32_t *ids, int32_t n_ids, float *logprobs,
                           int32_t *ranks, float *entropy, int32_t top_k, int32_t *top_ids, float *top_logprobs);

#ifdef __cplusplus
}
#endif

#endif /* QW_H */
