/*
 * scute.h - C ABI of the normal-form batched adapter layer on MI355X (gfx950).
 *
 * The layer computes, for every token t of a batch whose tokens belong to
 * many adapters a = a(t) over one shared base weight W,
 *
 *   y_t = ((x_t R_a) W) (.) s_a + b_a + sum_k c_k (((x_t A_k) (.) d_k) B_k (.) e_k)
 *
 * (row vectors; "The big picture: six extra slots in the LoRA computation",
 * paper-daily.com explainer of "Scute: Exact Batched Serving for PEFT
 * Adapters Beyond LoRA"). LoRA, DoRA, (IA)^3, VeRA and OFT adapters are all
 * written in this normal form ("What problem is it solving?").
 *
 * Buffer conventions (PyTorch nn.Linear layout; the formula uses transposes):
 *   x     [n][d_in]    activation dtype, row-major
 *   W     [d_out][d_in] activation dtype, row-major (K contiguous)
 *   y     [n][d_out]   float32
 *   A     [rank][d_in]   B [d_out][rank]
 *   A_sh  [r_v][d_in]    B_sh [d_out][r_v]
 *   Q, R  [d_in/blk][blk][blk], block kb maps input i -> output j via
 *         out[kb*blk + j] = sum_i in[kb*blk + i] * M[kb][i][j]
 *
 * Errors: every call returns a scute_status; 0 is success. On failure a
 * thread-local message is available from scute_last_error() and the object
 * passed in is left as it was (still usable). No C++ exception crosses this
 * boundary. Device-side faults of asynchronous calls surface at the caller's
 * next synchronisation of the stream.
 *
 * Threading: one layer may run forwards on one stream at a time. Loads and
 * unloads must not overlap a forward on the same layer; the caller
 * serialises them.
 */
#ifndef SCUTE_H
#define SCUTE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t scute_status;

#define SCUTE_OK 0
#define SCUTE_E_INVALID (-1)     /* null pointer or bad argument value        */
#define SCUTE_E_SHAPE (-2)       /* sizes inconsistent with the layer         */
#define SCUTE_E_NOMEM (-3)       /* allocation failed or capacity exhausted   */
#define SCUTE_E_HIP (-4)         /* HIP runtime error                         */
#define SCUTE_E_STATE (-5)       /* wrong state: id occupied / not loaded,
                                    stale plan, shared VeRA pair not set      */
#define SCUTE_E_UNSUPPORTED (-6) /* valid request this build does not serve   */

typedef enum scute_dtype {
  SCUTE_F32 = 0,
  SCUTE_BF16 = 1, /* stored as uint16 bit patterns */
  SCUTE_F64 = 2
} scute_dtype;

typedef enum scute_method {
  SCUTE_LORA = 0,       /* y = xW + b + c (xA) B                                 */
  SCUTE_DORA = 1,       /* y = x W_D + b, W_D = (W + cAB) diag(m / colnorm(W+cAB)) */
  SCUTE_IA3 = 2,        /* y = (xW) (.) l + b  (l on the s slot)                 */
  SCUTE_VERA = 3,       /* y = xW + b + (((x A_sh) (.) d) B_sh) (.) (c e)        */
  SCUTE_OFT = 4,        /* y = (x R) W + b, R = blockdiag(Cayley(Q_k))           */
  SCUTE_NORMAL_FORM = 5 /* slots given directly: R, s, b, one own term, VeRA term */
} scute_method;

typedef struct scute_layer scute_layer;
typedef struct scute_batch scute_batch;

/*
 * One adapter as it comes from its method ("How does Scute plug into vLLM?":
 * the converter rewrites each checkpoint in the normal form at load).
 * Every array is a HOST pointer in `dtype` (SCUTE_F64, SCUTE_F32, or
 * SCUTE_BF16 as uint16). Arrays a method does not use are ignored; an
 * optional array left null takes its identity value (ones, zero, identity).
 */
typedef struct scute_adapter_desc {
  int32_t method; /* scute_method                                            */
  int32_t dtype;  /* element type of the host arrays below                   */
  int32_t rank;   /* rank r of the own low-rank term (LoRA, DoRA, NORMAL_FORM
                     with A and B); 0 = no own term                          */
  int32_t blk;    /* block size of Q (OFT) or R (NORMAL_FORM); divides d_in  */
  double c;       /* scalar c: of the own term (LoRA, DoRA, NORMAL_FORM), or
                     of the shared term (VeRA; the pages' VeRA uses c = 1)   */
  const void* A;  /* [rank][d_in]   own down factor                          */
  const void* B;  /* [d_out][rank]  own up factor                            */
  const void* d;  /* [rank]   NORMAL_FORM own-term d (null: ones)            */
  const void* e;  /* [d_out]  NORMAL_FORM own-term e (null: ones)            */
  const void* m;  /* [d_out]  DoRA learned column lengths                    */
  const void* l;  /* [d_out]  (IA)^3 vector                                  */
  const void* vd; /* [r_v]    VeRA d (VERA; NORMAL_FORM shared term)         */
  const void* ve; /* [d_out]  VeRA e                                         */
  const void* Q;  /* [d_in/blk][blk][blk] OFT skew-symmetric blocks          */
  const void* R;  /* [d_in/blk][blk][blk] NORMAL_FORM rotation blocks        */
  const void* s;  /* [d_out]  NORMAL_FORM s (null: ones)                     */
  const void* b;  /* [d_out]  shift b, any method (null: zero)               */
} scute_adapter_desc;

/* Per-batch algorithmic cost (the byte / FLOP model; "Where is the cheapest
 * place to compute the remaining slots?": adapter work is priced in bytes,
 * added time = extra bytes / bandwidth + extra launches x launch cost). */
typedef struct scute_cost {
  double bytes;         /* x + W + y + every touched adapter's stored factors
                           + shared VeRA pair once if any VeRA row           */
  double adapter_bytes; /* bytes minus x, W and y                            */
  double flops;         /* 2 n d_in d_out + own terms + VeRA terms + rotations */
  double base_flops;    /* 2 n d_in d_out                                    */
  int32_t launches;     /* kernel launches per forward                       */
  int32_t n_tokens;
  int32_t n_segments;   /* runs of one adapter after the stable sort         */
  int32_t n_rot_rows;   /* rows with a rotation slot (OFT)                   */
  int32_t n_vera_rows;  /* rows with a shared VeRA term                      */
  int32_t n_touched;    /* distinct adapters with at least one token         */
  /* the same bytes split by the step that needs them (x counted in both):  */
  double gemm_bytes;     /* base GEMM + expand: x, W, y, B', s, b, VeRA e, B_sh */
  double prologue_bytes; /* rotation + shrink: x, A', P, VeRA d, A_sh          */
  /* the flops split the same way:                                           */
  double gemm_flops;     /* 2 n d_in d_out + expands (t B', u B_sh)           */
  double prologue_flops; /* shrinks (x A', x A_sh) + rotations (x P)          */
} scute_cost;

/* Create a layer context for one (d_in, d_out, activation dtype, device).
 * device >= 0: HIP device ordinal; every forward runs there.
 * device == -1: host-only context (fold, plan and cost model only; the
 *   forward returns SCUTE_E_UNSUPPORTED). Used to test host logic without a
 *   GPU.
 * act_dtype: SCUTE_BF16 (bf16 inputs, fp32 accumulate) or SCUTE_F32.
 * max_adapters: adapter ids run 0 .. max_adapters-1.
 * The library owns everything it allocates; release with scute_layer_destroy. */
scute_status scute_layer_create(int32_t device, int64_t d_in, int64_t d_out,
                                int32_t act_dtype, int32_t max_adapters,
                                scute_layer** out);

/* Free the layer and every adapter it holds. The caller must have
 * synchronised every stream that used it. Plans built for it become invalid
 * and must still be destroyed. Null is accepted. */
scute_status scute_layer_destroy(scute_layer* layer);

/* Set the shared VeRA pair ("Which slots can be merged at load?": VeRA's A
 * and B are shared by every VeRA tenant, so d and e stay live; "How does
 * Scute plug into vLLM?": VeRA keeps a reference to the shared matrices).
 * A_sh [r_v][d_in] and B_sh [d_out][r_v] are DEVICE pointers in the
 * activation dtype, BORROWED: the caller keeps them alive and unchanged
 * while the layer is used. Must precede loading any adapter with a VeRA
 * term; may be replaced only while no VeRA adapter is loaded.
 * Host-only layers accept host pointers (not dereferenced). */
scute_status scute_set_vera_shared(scute_layer* layer, const void* A_sh,
                                   const void* B_sh, int32_t r_v);

/* Load adapter `id`: fold its slots ("Which slots can be merged at load?":
 * a slot next to a factor the adapter owns merges into it, a slot next to
 * shared W or the shared VeRA pair stays live), in fp64 on the host, then
 * store the folded factors in library-owned device memory:
 *   own term:  A' = c A diag(d), B' = B diag(e)  (activation dtype)
 *   DoRA:      s = m / colnorm(W + cAB) stays live on the base path and
 *              also folds into B' (e = s), c folds into A'
 *   (IA)^3:    s = l live     VeRA: d, c e live     OFT: P = R - I
 *   s, b, VeRA d and e are stored in float32.
 * W_host ([d_out][d_in] in desc->dtype, HOST pointer) is read only for
 * DoRA and may be null otherwise. `stream` orders the uploads (null: the
 * default stream); the call returns after they complete.
 * Errors: SCUTE_E_STATE if `id` is occupied or the VeRA pair is missing,
 * SCUTE_E_SHAPE for a bad rank / block size, SCUTE_E_INVALID for a missing
 * array, SCUTE_E_NOMEM if device memory runs out. */
scute_status scute_load_adapter(scute_layer* layer, int32_t id,
                                const scute_adapter_desc* desc,
                                const void* W_host, void* stream);

/* Split the layer's output columns into n_proj projections (at most 4) that
 * share x and are computed by one GEMM over the stacked weight, e.g. q, k
 * and v ("How does Scute plug into vLLM?", paper-daily.com explainer of
 * "Scute: Exact Batched Serving for PEFT Adapters Beyond LoRA": OFT gives
 * each projection its own input rotation, which is why Scute splits the
 * q / k / v GEMM when OFT is present; with this call one GEMM keeps them).
 * col_end[i] (HOST array) is the end column of projection i: increasing,
 * every end but the last a multiple of 64, the last equal to d_out.
 * Only while no adapter is loaded (SCUTE_E_STATE otherwise); plans built
 * before become stale. n_proj = 1 with col_end[0] = d_out undoes it.
 * Errors: SCUTE_E_SHAPE for bad ends or n_proj, SCUTE_E_INVALID for null. */
scute_status scute_layer_set_projections(scute_layer* layer, int32_t n_proj,
                                         const int64_t* col_end);

/* Load adapter `id` like scute_load_adapter, with one rotation per
 * projection of the layer: desc->method must be SCUTE_NORMAL_FORM with
 * desc->R null, and R_proj[p] (HOST pointer, [d_in/blk][blk][blk] in
 * desc->dtype, blk = desc->blk) is the rotation of projection p's input;
 * a null R_proj[p] is the identity. Output columns of projection p compute
 * ((x R_p) W) (.) s + b + the adapter's terms. Each P_p = R_p - I is stored
 * like the single rotation slot, the n_proj of them one after another
 * (scute_read_slot of SCUTE_SLOT_P returns n_proj d_in blk elements).
 * Batches with such rows run the two-launch decode path (bf16, up to 256
 * rows), the prefill path (bf16, when every projection ends on a multiple
 * of 256) or the generic kernels (so does scute_layer_forward_noalloc).
 * Errors: SCUTE_E_STATE if the layer has one projection or `id` is
 * occupied, SCUTE_E_INVALID for another method, a non-null desc->R or a
 * null R_proj, SCUTE_E_SHAPE for a bad block size; otherwise as
 * scute_load_adapter. */
scute_status scute_load_adapter_proj(scute_layer* layer, int32_t id,
                                     const scute_adapter_desc* desc,
                                     const void* const* R_proj,
                                     const void* W_host, void* stream);

/* Unload adapter `id` and free its memory after `stream` drains.
 * SCUTE_E_STATE if `id` is not loaded. Plans built before become stale. */
scute_status scute_unload_adapter(scute_layer* layer, int32_t id, void* stream);

/* Build the batch plan from a HOST array token_adapter[n] (-1: base path
 * only): a stable sort of tokens by adapter so that every run of rows
 * belongs to one adapter ("Where is the cheapest place...": each tile of
 * the expand belongs to one adapter; each row looks up its tenant's VeRA
 * vectors and rotation). Rows with a rotation slot come first, then rows
 * with a shared VeRA term, then the rest, each group ordered by adapter id
 * and token index. The plan is library-owned, sized workspaces included,
 * and may be reused for any number of forwards with the same assignment
 * until the layer's adapters change. n may be 0.
 * Errors: SCUTE_E_STATE if a token names an id that is not loaded. */
scute_status scute_plan_batch(scute_layer* layer, const int32_t* token_adapter,
                              int32_t n, void* stream, scute_batch** out);

/* Plan flags for scute_plan_batch_flags. */
typedef enum scute_plan_flag {
  /* every forward with the plan gives the same bits for the same inputs:
   * decode-size batches run the fused MFMA path, whose K slices and shrink
   * slices are added in a fixed order with no float atomics (the other
   * paths already add in a fixed order) */
  SCUTE_PLAN_DETERMINISTIC = 1,
  /* Route variants of the two-launch decode path, for the route comparison
   * and time model of "Where is the cheapest place to compute the remaining
   * slots?" (the default route fuses every step into the GEMM's prologue and
   * epilogue). Any of them plans the batch on that path (SCUTE_E_UNSUPPORTED
   * if it does not take the batch); results equal the default route's up to
   * the order of fp32 additions. */
  /* the GEMM writes x W only; s (applied inside the pass), b and the own
   * low-rank term follow in an expand pass, the VeRA term in its own pass */
  SCUTE_PLAN_ROUTE_EXPAND_PASS = 2,
  /* with EXPAND_PASS: s applied by a pass of its own before the expand
   * (s copied to every row, then multiplied into the output) */
  SCUTE_PLAN_ROUTE_SEPARATE_S = 4,
  /* the VeRA term in a pass of its own after the GEMM (whole batch, the
   * shared B_sh read once per 32 VeRA rows) */
  SCUTE_PLAN_ROUTE_VERA_PASS = 8,
  /* the OFT rotation in a pass of its own before the prologue */
  SCUTE_PLAN_ROUTE_ROTATE_PASS = 16
} scute_plan_flag;

/* scute_plan_batch with flags (a bitwise or of scute_plan_flag; 0 gives
 * scute_plan_batch). Errors as scute_plan_batch, plus SCUTE_E_INVALID for an
 * unknown flag bit, SEPARATE_S without EXPAND_PASS, or DETERMINISTIC with a
 * route bit, and SCUTE_E_UNSUPPORTED when a route bit is set and the batch
 * does not fit the two-launch decode path. */
scute_status scute_plan_batch_flags(scute_layer* layer, const int32_t* token_adapter,
                                    int32_t n, uint32_t flags, void* stream,
                                    scute_batch** out);

/* Free a plan (after the streams that used it are synchronised). Null ok.
 * The plan records its device when it is built, so it may be freed before
 * or after its layer. */
scute_status scute_batch_destroy(scute_batch* batch);

/* The forward pass on `stream` (null: default stream), asynchronous.
 * x [n][d_in] and W [d_out][d_in] are DEVICE pointers in the activation
 * dtype; y [n][d_out] is a DEVICE float32 pointer that is fully written.
 * All three are borrowed for the call. Every step runs in this library's
 * HIP kernels: OFT rotation, base GEMM with the s / b epilogue, own-term
 * shrink and expand, and the whole-batch shared VeRA term ("How does Scute
 * plug into vLLM?": four steps, the rotation before the GEMM).
 * Range: inputs must be finite; every intermediate (rotation, shrink
 * sums, GEMM partials, expand) is held in float32 (the shrink sums and
 * rotation output are rounded to the activation dtype once as MFMA
 * operands), so any input scale whose products and sums stay inside the
 * float32 range is served; there is no fixed-point stage.
 * May be captured into a graph, and replayed between other forwards of the
 * plan; a plan's workspaces serve one forward at a time. From a decode plan's
 * first capture on each of its forwards, captured or not, makes one launch more,
 * which clears what the last one left (scute_cost.launches counts it).
 * Errors: SCUTE_E_STATE if the plan is stale or from another layer,
 * SCUTE_E_UNSUPPORTED on a host-only layer, SCUTE_E_INVALID for null or
 * misaligned pointers (16-byte alignment required). */
scute_status scute_layer_forward(scute_layer* layer, const scute_batch* batch,
                                 const void* x, const void* W, float* y,
                                 void* stream);

/* Bytes of the static device scratch that scute_layer_forward_noalloc uses
 * (one copy per device, held until the process ends). */
#define SCUTE_NOALLOC_SCRATCH_BYTES (16u << 20)

/* The forward for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * it needs no plan and allocates nothing. token_adapter is a DEVICE int32
 * array [n] (-1: base path only); x, W and y are as in scute_layer_forward.
 * The batch runs in token order on the generic kernels (the same arithmetic
 * as scute_layer_forward's generic path); the rotation output and shrink
 * sums live in the library's static scratch of SCUTE_NOALLOC_SCRATCH_BYTES
 * on the layer's device, which holds n * d_in * dtype_size (only when a
 * loaded adapter rotates) + n * max loaded rank * 4 + n * r_v * 4 (only when
 * a VeRA adapter is loaded) bytes, each part rounded up to 256. Every call on
 * a device shares that scratch and overwrites what it reads, so calls that
 * overlap on one device race: order them on one stream. Ids are checked on
 * the device: a row whose id is out of range or not loaded gets NaN.
 * Errors: SCUTE_E_SHAPE if n is outside [0, 65535] or the batch needs more
 * scratch than there is; SCUTE_E_INVALID for null or misaligned pointers
 * (16-byte x, W, y; 4-byte token_adapter); SCUTE_E_STATE if a VeRA adapter
 * is loaded and the shared pair is not set; SCUTE_E_UNSUPPORTED on a
 * host-only layer or a device index past 63. An adapter loaded with
 * scute_load_adapter_proj makes the rotation output one block of n rows
 * per projection (counted in the scratch a batch needs). */
scute_status scute_layer_forward_noalloc(scute_layer* layer, const int32_t* token_adapter,
                                         int32_t n, const void* x, const void* W, float* y,
                                         void* stream);

/* The FFN gate after the up projection: h = silu(g) (.) u element-wise, with
 * silu(z) = z / (1 + exp(-z)), the gate activation of the Llama models the
 * pages evaluate on. (IA)^3 multiplies the FFN intermediate
 * sigma(x W_g) (.) (x W_u) by l; products reorder, so l is the s slot of the
 * up projection ("The big picture: six extra slots in the LoRA
 * computation"), u is that layer's output and g the gate projection's.
 * g, u, h: DEVICE float32 arrays of `count` elements, h may be u; 16-byte
 * aligned. Errors: SCUTE_E_INVALID for null or misaligned pointers or
 * count < 0; SCUTE_E_HIP if the launch fails. */
scute_status scute_silu_gate(const float* g, const float* u, float* h, int64_t count, void* stream);

/* ---- between the adapter layers of a decoder block ----------------------- */

/* The operators that run from the q / k / v layer's output to the output
 * projection's input and from one block's output to the next layer's x. They
 * belong to no layer: each names its device, launches on `stream` (null: that
 * device's default stream) with that device current, allocates nothing, keeps
 * nothing between calls and may be captured into a graph. Pointers are DEVICE
 * pointers on that device, borrowed for the call, and outputs overlap no
 * input or other output unless stated (SCUTE_E_INVALID where the addresses show
 * it). Every call checks its arguments before it touches the device. */

/* A paged key-value cache: n_pages pages of page_size positions. Element
 * (page p, position i of the page, head g, dim j) of K and of V lies
 * p page_stride + i token_stride + g head_stride + j elements from k and v
 * (so [page][position][head][dim] and [page][head][position][dim] are both
 * served). A slot names one position of the cache: page * page_size + i. */
typedef struct scute_kv_cache {
  int32_t device;
  int32_t dtype;      /* SCUTE_BF16 or SCUTE_F32                             */
  int32_t page_size;  /* positions of a page, 1 .. 65536                     */
  int32_t n_kv_heads; /* 1 .. 1024                                           */
  int32_t head_dim;   /* a multiple of 8, 8 .. 256                           */
  int32_t reserved;   /* 0                                                   */
  int64_t n_pages;    /* 1 .. 2^31 - 1                                       */
  int64_t page_stride, token_stride, head_stride; /* multiples of 8, 8 .. 2^40
                         (token_stride below 2^24)                           */
  void* k;            /* 16-byte aligned                                     */
  void* v;
} scute_kv_cache;

/* Pages and slots of one step's tokens from the requests' lengths, without
 * the host: request r holds old_len[r] positions of the cache, its pages in
 * table[r][0 .. ceil(old_len[r] / page_size)); it brings new_len[r] tokens
 * (0: none), or ends (new_len[r] < 0). The free pages lie in a ring of
 * ring_size entries from cursor[0] (head) up to cursor[1] (tail), both
 * counted on without wrapping (entry c is ring[c mod ring_size]).
 *   - In the requests' order each takes the pages its new positions need from
 *     the head of the ring into its row of the table. A request gets all of
 *     them or none: when the free pages do not suffice, or its pages would
 *     pass the table's width, it is refused and keeps old_len; those after it
 *     that need pages are refused too when the ring ran out.
 *   - The pages of a request that ends go back to the tail of the ring and
 *     may be taken from the next step on; its row of the table is left as
 *     it is.
 * Tokens stand in the requests' order. Token t of a request's new tokens gets
 * its position (len - 1 = pos), its request, and its slot; tokens of a refused
 * request and every row past the last token up to max_tokens get slot -1,
 * request -1, pos 0 and len 0, which the operators below skip, so a captured
 * step may hold fewer tokens than rows.
 * Lengths, token and page totals may be at most 2^30, new lengths 2^29;
 * negative old lengths count as 0; the cursors count from 0 up. Errors:
 * SCUTE_E_INVALID for null or misaligned pointers, an output that is also an
 * input or an unknown flag, SCUTE_E_SHAPE for sizes out of range. */
typedef enum scute_assign_flag {
  /* a request is refused, and keeps old_len, when one of its tokens has no row
   * (its tokens and those of the requests before it are more than max_tokens);
   * those after it that bring tokens are then refused too. Without the flag
   * such a request is placed: tokens past the last row have pages and count in
   * seq_len, and nothing of them can be stored, so it is the caller who sees to
   * cu_len[n_requests] <= max_tokens */
  SCUTE_ASSIGN_FIT_ROWS = 1,
  /* row r is request r's: its one token, or nothing (slot -1) where it brings
   * none, ends or is refused, so that a row keeps its request from step to step
   * (cu_len[r] is r). A request that brings more than one token is refused.
   * max_tokens is n_requests or more (SCUTE_E_SHAPE otherwise) */
  SCUTE_ASSIGN_ONE_EACH = 2
} scute_assign_flag;

typedef struct scute_cache_assign_args {
  int32_t device;
  int32_t n_requests;   /* 0 .. 65536                                        */
  int32_t table_width;  /* pages of a request at most, 1 .. 2^24             */
  int32_t page_size;    /* 1 .. 65536                                        */
  int32_t ring_size;    /* 1 .. 2^30                                         */
  int32_t max_tokens;   /* rows of slot, req, pos and len, 0 .. 2^30         */
  int64_t table_stride; /* entries between rows of the table, >= table_width */
  const int32_t* old_len; /* [n_requests]                                    */
  const int32_t* new_len; /* [n_requests]                                    */
  int32_t* table;         /* [n_requests][table_stride], updated             */
  int32_t* ring;          /* [ring_size], updated                            */
  const int64_t* cursor;  /* [2] head, tail                                  */
  int64_t* cursor_out;    /* [2] head and tail after the step                */
  int32_t* seq_len;       /* [n_requests] positions held after the step (0:
                             the request ended)                              */
  int32_t* cu_len;        /* [n_requests + 1] first token of each request,
                             and the tokens in all                           */
  int64_t* slot;          /* [max_tokens]                                    */
  int32_t* req;           /* [max_tokens]                                    */
  int32_t* pos;           /* [max_tokens]                                    */
  int32_t* len;           /* [max_tokens]                                    */
  int32_t* counts;        /* [4] tokens placed, pages taken, requests refused,
                             pages returned                                  */
  uint32_t flags;         /* a bitwise or of scute_assign_flag               */
  uint32_t reserved;      /* 0                                               */
} scute_cache_assign_args;

scute_status scute_cache_assign(const scute_cache_assign_args* args, void* stream);

/* Requests that go on from others, without the host. Request r holds, after
 * the call, the first keep[r] positions of what request parent[r] held before
 * it (itself: kept or cut back; another: samples of one prompt, beams; a parent
 * outside 0 .. n_requests - 1: the request ends), n = min(len[parent], keep)
 * of them, at most table_width page_size. len[r] positions were held, their
 * pages in table[r]; entries outside 0 .. n_pages - 1 hold no page.
 *   - Whole pages are shared: table_out[r] names the parent's.
 *   - The last page, where n does not fill it, is written next, so it must be
 *     its request's alone: of the requests that hold it partly the first keeps
 *     it, when none holds it wholly; each of the others takes a page from the
 *     head of the ring, in the requests' order, and src[r], dst[r], n[r] say
 *     which page's first n positions to copy where (scute_cache_copy, for each
 *     layer's cache; -1, -1, 0: nothing). Where the free pages run out a
 *     request is refused: it keeps its whole pages, and seq_len[r] says so.
 *   - window > 0: a page whose positions all lie in [sinks, n - window) is
 *     dropped (table_out -1), as rows from n on do not see it
 *     (scute_sink_attention with this window and these sinks). A refused
 *     request's pages are dropped by the n it did not get: where the window is
 *     not whole pages, rows from its seq_len[r] on may see the end of one that is
 *     gone, so such a request ends, or is read again from its start.
 *   - Pages that some request held and none holds any more go to the tail of
 *     the ring in ascending order, and may be taken from the next step on.
 * Entries of table_out past a request's pages are -1. The table that is handed
 * in stays as it is, and table_out may not overlap it. Requests that share
 * pages, or have dropped some, end here: scute_cache_assign gives back every
 * entry of a request that ends there.
 * Lengths and cursors as in scute_cache_assign. workspace: at least what
 * scute_cache_fork_workspace says, 256-byte aligned, zeroed once before its
 * first use (calls of any sizes may use it in turn); calls that may overlap in time need workspaces of their own.
 * Errors: as scute_cache_assign's; SCUTE_E_INVALID for a workspace that is too
 * small. */
typedef struct scute_cache_fork_args {
  int32_t device;
  int32_t n_requests;   /* 0 .. 65536                                        */
  int32_t table_width;  /* 1 .. 2^24                                         */
  int32_t page_size;    /* 1 .. 65536                                        */
  int32_t ring_size;    /* 1 .. 2^30                                         */
  int32_t n_pages;      /* pages of the cache, 1 .. 2^24                     */
  int32_t window;       /* 0: no page is dropped                             */
  int32_t sinks;        /* >= 0                                              */
  int64_t table_stride, table_out_stride; /* >= table_width                  */
  const int32_t* len;     /* [n_requests]                                    */
  const int32_t* parent;  /* [n_requests]                                    */
  const int32_t* keep;    /* [n_requests], null: all                         */
  const int32_t* table;   /* [n_requests][table_stride]                      */
  int32_t* ring;          /* [ring_size], updated                            */
  const int64_t* cursor;  /* [2] head, tail                                  */
  int64_t* cursor_out;    /* [2]                                             */
  int32_t* table_out;     /* [n_requests][table_out_stride]                  */
  int32_t* seq_len;       /* [n_requests] positions held after the call      */
  int32_t* src;           /* [n_requests] page to copy from                  */
  int32_t* dst;           /* [n_requests] page to copy to                    */
  int32_t* n;             /* [n_requests] positions to copy                  */
  int32_t* counts;        /* [4] requests that hold positions, pages taken,
                             requests refused, pages returned                */
  void* workspace;
  int64_t workspace_bytes;
} scute_cache_fork_args;

scute_status scute_cache_fork_workspace(int32_t n_requests, int32_t n_pages, int64_t* bytes);
scute_status scute_cache_fork(const scute_cache_fork_args* args, void* stream);

/* Copy the first n[i] positions (at most a page's) of page src[i] to page
 * dst[i], K and V, for i in 0 .. n_copies - 1 (device arrays). An entry whose
 * pages are the same or outside the cache, or whose n is not positive, copies
 * nothing. No page may be written by two entries, or be read by one and written by another.
 * Errors: SCUTE_E_INVALID for null or misaligned pointers, SCUTE_E_SHAPE for
 * n_copies outside 0 .. 2^20. */
scute_status scute_cache_copy(const scute_kv_cache* cache, const int32_t* src, const int32_t* dst,
                              const int32_t* n, int32_t n_copies, void* stream);

/* Positions that stay, moved together: of request r, place start[r] + j gets
 * what position kept[r][j] held before the call, K and V, for j below n_kept[r]
 * (at most kept_width), so the request then holds new_len[r] = start[r] +
 * n_kept[r] positions (scute_cache_fork with keep = new_len gives the pages
 * behind them back). A position only moves down: where kept[r][j] lies before
 * its new place, or either lies past the table or on a page outside the cache,
 * the place keeps what it held. Ascending positions always move down.
 * The pages that are written may not be another request's too. Several layers'
 * caches are compacted by a call each. start below 0 counts as 0.
 * table [n_requests][table_stride], kept [n_requests][kept_stride], new_len
 * null or [n_requests] (start + n_kept saturates at 2^30).
 * Errors: SCUTE_E_INVALID for null or misaligned pointers or a new_len that is
 * an input, SCUTE_E_SHAPE for sizes out of range. */
scute_status scute_cache_compact(const scute_kv_cache* cache, const int32_t* table, int64_t table_stride,
                                 int32_t n_requests, int32_t table_width, const int32_t* start,
                                 const int32_t* kept, int64_t kept_stride, int32_t kept_width,
                                 const int32_t* n_kept, int32_t* new_len, void* stream);

/* Rotary positions: pair i of a head's first rot_dim elements is turned by
 * the angle pos[axis[i]][t] * freq[i] (one axis for text; time, height and
 * width for images and video). The angle is reduced in 64 bits, so far
 * positions lose nothing. Elements past rot_dim stay as they are. */
typedef struct scute_rotary {
  int32_t head_dim;
  int32_t rot_dim;      /* even, 0 .. head_dim                               */
  int32_t n_axes;       /* 1 .. 8                                            */
  int32_t interleaved;  /* 0: pair i is (i, i + rot_dim / 2); 1: (2i, 2i + 1) */
  const double* freq;   /* [rot_dim / 2] radians a position                  */
  const int32_t* axis;  /* [rot_dim / 2] axis of each pair, 0 .. n_axes - 1
                           (others count as axis 0); null: all axis 0        */
} scute_rotary;

/* Rotate q and k of n_tokens tokens, store k and v in the cache. q
 * [n_tokens][n_heads][head_dim], k and v [n_tokens][n_kv_heads][head_dim] in
 * src_dtype (SCUTE_F32: a layer's y, each a range of its columns; or
 * SCUTE_BF16), their rows q_stride, k_stride and v_stride elements apart.
 * pos [n_axes][n_tokens], its axes pos_stride elements apart. slot
 * [n_tokens]: a token whose slot is negative or past the cache is not
 * stored; slots that repeat leave one of their tokens, whichever. q_out
 * [n_tokens][n_heads][head_dim] in the cache's type, its rows q_out_stride
 * apart; it may be q itself where type and stride are the same. Products are fp32, rounded once to the cache's type.
 * Errors: SCUTE_E_INVALID for null or misaligned pointers (each to its
 * element) or a bad dtype, SCUTE_E_SHAPE for sizes out of range. */
scute_status scute_rotary_store(const scute_rotary* rotary, const scute_kv_cache* cache, const void* q,
                                int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, int32_t src_dtype, const int32_t* pos,
                                int64_t pos_stride, const int64_t* slot, int32_t n_tokens,
                                int32_t n_heads, void* q_out, int64_t q_out_stride, void* stream);

/* Norms of the heads of q and of k, each over a head's head_dim elements,
 *   N(v) = v / sqrt(mean(v^2) + eps) (.) w + b (SCUTE_NORM_RMS)
 * or the same of v - mean(v) (SCUTE_NORM_LAYER). */
typedef struct scute_head_norm {
  int32_t kind;       /* SCUTE_NORM_RMS (0) or SCUTE_NORM_LAYER (1)           */
  float eps;
  const float* q_w;   /* [head_dim], or of each head; null: ones (weights),   */
  const float* q_b;   /* zeros (biases)                                       */
  const float* k_w;
  const float* k_b;
  int32_t q_stride;   /* elements between the heads' vectors: 0 where all     */
  int32_t k_stride;   /* heads have the same, head_dim or more otherwise      */
} scute_head_norm;

/* scute_rotary_store with norms of the heads of q and k before the rotation,
 * in the same pass: N(q) and N(k) are rotated, v is stored as it is. All of it
 * is fp32 and rounded once, to the cache's type (squares whose sum passes fp32
 * give the biases alone; the variance is summed about the mean). Arguments and
 * errors as there, and SCUTE_E_INVALID for a kind or a vector's address that is
 * not one, SCUTE_E_SHAPE for a stride between 1 and head_dim - 1, below 0 or past 2^20. */
scute_status scute_norm_rotary_store(const scute_rotary* rotary, const scute_head_norm* norm,
                                     const scute_kv_cache* cache, const void* q, int64_t q_stride,
                                     const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                     int32_t src_dtype, const int32_t* pos, int64_t pos_stride,
                                     const int64_t* slot, int32_t n_tokens, int32_t n_heads, void* q_out,
                                     int64_t q_out_stride, void* stream);

/* Bytes of workspace that scute_paged_attention may use on `device` for
 * heads of head_dim elements. */
scute_status scute_paged_attention_workspace(int32_t device, int32_t head_dim, int64_t* bytes);

/* Attention of new tokens over the paged cache. Row i belongs to request
 * req[i] (null: request i) and sees that request's positions
 * max(0, n - window) .. n - 1 (window 0: all of them), with n = len[i] or, where
 * that is less, what a row of the table can hold (table_width page_size, and
 * 2^29); position t lies in page table[request][t / page_size].
 *   out[i][h] = sum_t softmax_t(scale q[i][h] . K[t][g]) V[t][g]
 * with g = h / (n_heads / n_kv_heads). A row that sees nothing (len <= 0, or a
 * request outside 0 .. n_requests - 1) gives zeros; positions whose page lies
 * outside the cache are not seen.
 * q and out [n_rows][n_heads][head_dim] in the cache's type, rows q_stride and
 * out_stride elements apart (multiples of 8, 16-byte aligned pointers).
 * Several rows of one request (its new tokens, each with its own length) are
 * several rows of one call; those that follow each other share the reads of
 * its cache. Scores, the softmax and the sums are fp32 (values whose sum over a
 * row's positions passes fp32 give infinities); the weights enter a
 * bf16 cache's products as sums of two bf16 values. A V that is not finite makes
 * those elements of the output not finite that see it, as the sum says: an
 * infinity stays one (where its weight is not 0 in fp32). The result depends on
 * the rows' requests and lengths only, never on the order in which work-groups
 * end.
 * workspace: `workspace_bytes` (at least what scute_paged_attention_workspace
 * says), 256-byte aligned, zeroed once by the caller before its first use;
 * every call leaves its counters zero. Calls that may overlap in time need
 * workspaces of their own.
 * Errors: SCUTE_E_INVALID for null or misaligned pointers, a workspace that
 * is too small, or a scale that is not finite (times log2(e) in fp32);
 * SCUTE_E_SHAPE for sizes out of range. */
scute_status scute_paged_attention(const scute_kv_cache* cache, const void* q, int64_t q_stride,
                                   int32_t n_heads, const int32_t* table, int64_t table_stride,
                                   int32_t n_requests, int32_t table_width, const int32_t* len,
                                   const int32_t* req, int32_t n_rows, float scale, int32_t window,
                                   void* out, int64_t out_stride, void* workspace,
                                   int64_t workspace_bytes, void* stream);

/* scute_paged_attention where the first `sinks` positions stay visible: row i
 * sees t < n with t < sinks or t >= n - window (window 0 or sinks 0: as there).
 * Positions between them are not read, and their pages need not be in the
 * cache (scute_cache_fork drops them). Arguments, workspace and errors as
 * there, and SCUTE_E_SHAPE for sinks below 0. */
scute_status scute_sink_attention(const scute_kv_cache* cache, const void* q, int64_t q_stride,
                                  int32_t n_heads, const int32_t* table, int64_t table_stride,
                                  int32_t n_requests, int32_t table_width, const int32_t* len,
                                  const int32_t* req, int32_t n_rows, float scale, int32_t window,
                                  int32_t sinks, void* out, int64_t out_stride, void* workspace,
                                  int64_t workspace_bytes, void* stream);

typedef enum scute_shared_flag {
  SCUTE_SHARED_ALWAYS = 1 /* shares however little that saves */
} scute_shared_flag;

/* Bytes of workspace that scute_shared_attention may use for calls of up to
 * max_rows rows in up to max_groups groups. Errors as for the call's sizes. */
scute_status scute_shared_attention_workspace(int32_t device, int32_t dtype, int32_t head_dim,
                                              int32_t n_heads, int32_t n_kv_heads, int32_t max_rows,
                                              int32_t max_groups, int64_t* bytes);

/* scute_paged_attention, without a window, of rows whose contexts begin with
 * the same positions: rows group[g] .. group[g + 1] - 1 (group [n_groups + 1],
 * ascending) are of requests that hold their first shared_len[g] positions in
 * the same pages (a prompt's samples, a system prompt's users), which are read
 * once for all of them, through the table of a row of the group that sees most
 * of them. A row sees its positions below len as there, shared or its own,
 * rows of no request or of length 0 nothing; rows of no group share nothing,
 * and shared_len may be 0. Results are those of scute_paged_attention but for
 * the order of the sums and a bf16 cache's weights, the sums of a value cut off to
 * bf16 and of the rest rounded to it (off by 2^-15 at most; an infinite V that a
 * row sees with a weight under 2^-100 may give NaN). Where sharing cannot save the
 * reads of 256 MiB (rows past one a group, at the table's whole width) the call is
 * scute_paged_attention's, unless flags says otherwise.
 * group and shared_len are device arrays; group is not checked: offsets that
 * do not ascend give rows whose output is not defined, no access out of bounds.
 * workspace as there, of at least what scute_shared_attention_workspace says
 * for n_rows and n_groups; one that is large enough may serve calls of any sizes
 * and caches of any head_dim in turn, scute_paged_attention's too. flags: a bitwise or of scute_shared_flag. Errors as
 * there, SCUTE_E_INVALID for an unknown flag, SCUTE_E_SHAPE for n_groups outside
 * 0 .. 65536 or more rows and heads than can be numbered at the table's whole width
 * (rows x key heads x tiles of 16 query heads x table positions / 32, or / 16 in
 * float32, stay under 2^31). */
scute_status scute_shared_attention(const scute_kv_cache* cache, const void* q, int64_t q_stride,
                                    int32_t n_heads, const int32_t* table, int64_t table_stride,
                                    int32_t n_requests, int32_t table_width, const int32_t* len,
                                    const int32_t* req, int32_t n_rows, const int32_t* group,
                                    const int32_t* shared_len, int32_t n_groups, float scale, void* out,
                                    int64_t out_stride, void* workspace, int64_t workspace_bytes,
                                    uint32_t flags, void* stream);

/* The norms around a block's residual:
 *   h' = h_scale h + y_scale (gate (.) N_post(y))     x = N_pre(h')
 * N(v) = v / sqrt(mean(v^2) + eps) (.) w + b (SCUTE_NORM_RMS), or the same of
 * v - mean(v) (SCUTE_NORM_LAYER). */
typedef enum scute_norm_kind { SCUTE_NORM_RMS = 0, SCUTE_NORM_LAYER = 1 } scute_norm_kind;

typedef struct scute_norm {
  int32_t device;
  int32_t kind;         /* scute_norm_kind                                   */
  int32_t d;            /* 1 .. 32768                                        */
  int32_t post;         /* 0: y enters as it is; 1: through N_post           */
  float eps;
  float h_scale, y_scale;
  int32_t reserved;     /* 0                                                 */
  const float* post_w;  /* [d] each, null: ones (weights), zeros (biases)    */
  const float* post_b;
  const float* pre_w;
  const float* pre_b;
} scute_norm;

/* y [n_rows][d] (a layer's output; null: h' = h_scale h), h [n_rows][d], gate
 * null, [d] (gate_stride 0) or [n_rows][d] float32; h_out [n_rows][d] in h's
 * type (null: not written; may be h itself), x [n_rows][d] (null: no N_pre).
 * Types SCUTE_F32 or SCUTE_BF16, rows *_stride elements apart. x is computed
 * from h' before it is rounded to h's type. Sums are fp32 (squares whose sum
 * passes fp32 give zeros); the variance is summed about the mean.
 * Errors: SCUTE_E_INVALID for null or misaligned pointers (each to its
 * element), a bad dtype, x that is also h, y or h_out, or neither output;
 * SCUTE_E_SHAPE for sizes out of range. */
scute_status scute_residual_norm(const scute_norm* norm, const void* y, int32_t y_dtype, int64_t y_stride,
                                 const void* h, int32_t h_dtype, int64_t h_stride, const float* gate,
                                 int64_t gate_stride, void* h_out, int64_t h_out_stride, void* x,
                                 int32_t x_dtype, int64_t x_stride, int32_t n_rows, void* stream);

/* Algorithmic bytes / FLOPs / launches of one forward with this plan. */
scute_status scute_cost_model(const scute_layer* layer, const scute_batch* batch,
                              scute_cost* out);

/* ---- introspection (tests, debugging) ---------------------------------- */

typedef enum scute_slot {
  SCUTE_SLOT_A = 0,  /* folded A' [rank8][d_in]       activation dtype */
  SCUTE_SLOT_B = 1,  /* folded B' [d_out][rank8]      activation dtype
                        (rank8: the rank rounded up to a multiple of 8;
                        the added rows of A' and columns of B' are zero) */
  SCUTE_SLOT_S = 2,  /* live s [d_out]                float32          */
  SCUTE_SLOT_BIAS = 3, /* b [d_out]                   float32          */
  SCUTE_SLOT_VD = 4, /* VeRA d [r_v]                  float32          */
  SCUTE_SLOT_VE = 5, /* VeRA e, c folded [d_out]      float32          */
  SCUTE_SLOT_P = 6   /* R - I [d_in/blk][blk][blk]    activation dtype
                        (kept transposed per block on the device;
                        scute_read_slot returns R - I itself)         */
} scute_slot;

typedef struct scute_adapter_info {
  int32_t loaded;
  int32_t method;
  int32_t rank;  /* stored rank: the own term's rank rounded up to 8 (0: none) */
  int32_t blk;
  int32_t has_R, has_s, has_b, has_term, has_vera;
} scute_adapter_info;

scute_status scute_adapter_info_get(const scute_layer* layer, int32_t id,
                                    scute_adapter_info* out);

/* Copy one stored slot of adapter `id` to HOST memory `dst` of `dst_bytes`
 * bytes (must be exactly the slot's size). SCUTE_E_STATE if the adapter
 * does not hold that slot. */
scute_status scute_read_slot(const scute_layer* layer, int32_t id, int32_t slot,
                             void* dst, int64_t dst_bytes);

typedef struct scute_batch_info {
  int32_t n;
  int32_t n_segments;
  int32_t n_rot_rows;  /* rows 0 .. n_rot_rows-1 of the sorted order rotate */
  int32_t n_vera_rows;
  int32_t max_rank;
  int32_t path;        /* kernels the forward will run: 0 generic, 1 MFMA decode, 2 MFMA prefill */
} scute_batch_info;

scute_status scute_batch_info_get(const scute_batch* batch, scute_batch_info* out);

/* Whether a forward of this plan had a cross-work-group wait give up
 * (*out = 1) since the plan was built or last reset (*out = 0 otherwise).
 * Only the fused decode path waits across work-groups; its waits are bounded
 * (about 2^20 polls) and a wait that gives up records the failure and lets
 * the kernel finish instead of hanging, so that forward's output is not
 * valid. Call after synchronising the stream the forwards ran on; the read
 * is a blocking device-to-host copy. reset != 0 clears the flag afterwards.
 * Errors: SCUTE_E_INVALID for null pointers, SCUTE_E_HIP if the copy fails.
 * Plans on other paths always report 0. */
scute_status scute_batch_wait_failures(const scute_batch* batch, int32_t reset, int32_t* out);

/* Copy the plan's tables to HOST memory:
 *   perm[n]            token index at each sorted position
 *   seg[3*n_segments]  (adapter id, first sorted position, length) per run
 * Either pointer may be null. */
scute_status scute_batch_read(const scute_batch* batch, int32_t* perm, int32_t* seg);

/* ---- kernel timing (instrumentation) ------------------------------------ */

/* When enabled, every forward on this layer records a HIP event pair around
 * each of its kernel launches, on the forward's stream. Timings accumulate
 * per kernel name until read. Costs a little launch overhead; off by default. */
scute_status scute_profile_enable(scute_layer* layer, int32_t enable);

typedef struct scute_kernel_time {
  char name[32];     /* kernel role, e.g. "gemm"                           */
  int32_t launches;  /* launches timed since the last read                 */
  double total_ms;   /* summed event-to-event time of those launches       */
} scute_kernel_time;

/* Wait for the recorded events, write up to `capacity` per-kernel totals to
 * HOST memory `out`, set *count to the number of kernel names, and reset
 * the totals. */
scute_status scute_profile_read(scute_layer* layer, scute_kernel_time* out, int32_t capacity,
                                int32_t* count);

/* Launch `count` empty kernels (one wave each) back to back on `stream`
 * (null: default stream) on the current device, for the launch-cost term of
 * the time model in "Where is the cheapest place to compute the remaining
 * slots?" (added time = extra bytes / bandwidth + extra launches x launch
 * cost): the caller times them with events. Errors: SCUTE_E_INVALID if
 * count < 0; SCUTE_E_HIP if a launch fails. */
scute_status scute_launch_empty(int32_t count, void* stream);

/* Thread-local message of the last failed call on this thread ("" if none). */
const char* scute_last_error(void);

/* Library version string. */
const char* scute_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SCUTE_H */
