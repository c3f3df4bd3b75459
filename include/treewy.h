/*
 * treewy.h -- C ABI of the TreeWY speculative-verification library for Gated
 * DeltaNet (GDN) layers on sm_103a (GB300).
 *
 * Method: "TreeWY: Speculative Verification for Gated DeltaNet Hybrids".
 * For one GDN layer, a batch of R requests, H value heads and one draft tree
 * per request, verification computes every draft node's output from the
 * committed state S0 without materialising a per-node state, and commit
 * rebuilds the one accepted state.
 *
 *   gated delta rule (paper §1 Eq. (1)):
 *       S_n = alpha_n S_par (I - beta_n k_n k_n^T) + beta_n v_n k_n^T,  o_n = S_n q_n
 *   pseudo-values U (paper §3 "Key rewrite" and Eq. (2)):
 *       (I + A) U = diag(beta) (V - diag(gamma) (S0 K^T)^T),
 *       A[n,i] = beta_n (gamma_n / gamma_i) (k_i . k_n) for i a strict ancestor of n,
 *       gamma_n = product of alpha over the root-to-n path, n included
 *   outputs (technical review §3.1 Eq. (5), restricted to ancestors as in §3.2):
 *       o_n = gamma_n S0 q_n + sum_{i ancestor of n or n} (gamma_n/gamma_i) (k_i . q_n) u_i
 *   commit (paper §3 "Reconstruct on commit", review Eq. (6)):
 *       S_a = gamma_a S0 + sum_{i on the root-to-a path} (gamma_a/gamma_i) u_i k_i^T
 *
 * Around it, for a server's pool of states: treewy_extend (the same rule over
 * a prompt's or a decode step's tokens), treewy_qk_norm (the normed q and k
 * that all of these read) and treewy_copy_slots (forking and compacting the
 * pool).  In the softmax layers between the GDN ones, treewy_attend verifies a
 * draft against a context kept in pages of 8 bits, treewy_append takes the
 * accepted path (or a prompt) into it, and treewy_add_norm adds the residual
 * and norms the rows of the next projection, in 8 bits where wanted.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All pointers in treewy_batch are DEVICE pointers to memory the caller
 *   owns; the library allocates no device memory and keeps no pointer after
 *   a call returns.  Calls are asynchronous on `stream` (0 = legacy default
 *   stream) and never synchronise the host.
 * - Errors the host can see (null pointers, unsupported sizes, misaligned
 *   buffers, launch failures) return a non-zero treewy_status before or at
 *   launch; treewy_last_error() then describes the problem.  Errors in the
 *   contents of device arrays (a parent index out of range, a tree larger
 *   than max_nodes, an accepted index outside the tree, a node range past T)
 *   cannot be seen by the host: the kernels set bits in status[r] for the
 *   request and skip it, leaving its outputs (or its state) untouched.
 * - Node rows: request r owns rows t = node_offset[r] .. node_offset[r+1]-1
 *   of every per-node array, node n of the request being row node_offset[r]+n.
 *   Nodes are in a topological order (every parent precedes its children;
 *   the pages use DFS pre-order, which is one such order).
 */
#ifndef TREEWY_H
#define TREEWY_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
typedef enum treewy_status {
  TREEWY_OK = 0,
  TREEWY_ERR_INVALID_ARG = 1,   /* null pointer, negative size, misalignment */
  TREEWY_ERR_UNSUPPORTED = 3,   /* sizes outside what the kernels implement */
  TREEWY_ERR_CUDA = 4           /* a CUDA runtime/driver call failed */
} treewy_status;

/* Bits of the per-request device status word.  Kernels only OR bits into
   status[r]; the caller zeroes the array before a round of calls. */
enum {
  TREEWY_STATUS_BAD_TREE = 1,       /* parent[n] outside [-1, n), or node range past T */
  TREEWY_STATUS_TOO_MANY_NODES = 2, /* N_r > max_nodes (or N_r < 0) */
  TREEWY_STATUS_BAD_ACCEPTED = 4,   /* accepted[r] outside [-1, N_r) (commit only) */
  TREEWY_STATUS_BAD_SLOT = 8,       /* state_slot[r] outside [0, num_slots) */
  TREEWY_STATUS_TIMEOUT = 16,       /* an internal wait gave up after ~1 s; that
                                       (request, head) was skipped */
  TREEWY_STATUS_COMMIT_REFUSED = 32, /* treewy_commit_verify only: the previous
                                       round's commit of this request was refused
                                       (its state is unchanged); the bits beside
                                       it say why */
  TREEWY_STATUS_BAD_POSITION = 64,  /* treewy_qk_norm: a position outside the
                                       rotation table */
  TREEWY_STATUS_SLOT_CLASH = 128,   /* treewy_copy_slots: the move's destination
                                       is written by another move too, or its
                                       source is another move's destination */
  TREEWY_STATUS_BAD_PAGE = 256      /* treewy_attend, treewy_append: a page index
                                       outside the pool, or a length that is
                                       negative or above what the call or the
                                       request's pages hold */
};

/* Element type of q, k and v. */
enum {
  TREEWY_DTYPE_BF16 = 0,
  TREEWY_DTYPE_F32 = 1
};

/* Flags. */
enum {
  /* Use the portable kernels (CUDA cores, no bulk tensor copies) even where
     the tensor-core verification (dk = dv = 128, bf16 q/k/v: warp-level
     MMAs for batches of trees of at most 32 nodes, tcgen05 above) or the
     bulk-copy commit (dk = dv = 128) applies.  Same results within rounding. */
  TREEWY_FLAG_FORCE_GENERIC = 1u,
  /* The state pool holds bf16 instead of f32: the dtype in which the GDN
     state is kept when serving (paper §2 "The memory problem": dv x dk x 2 B
     per head), half the bytes of every state read and write.  Verification
     takes the bf16 S0 as exact values; commit forms S_a in f32 and stores it
     rounded to nearest (ties to even) bf16, so each committed element is
     within 2^-8 of its relative value.  The storeall comparator entry points
     reject this flag with TREEWY_ERR_UNSUPPORTED. */
  TREEWY_FLAG_STATE_BF16 = 2u
};

/* Largest draft tree per request. */
#define TREEWY_MAX_NODES 64

/*
 * One GDN layer's worth of draft-tree data.
 *
 * Sizes: R >= 0 requests, H >= 1 value heads, key/value head sizes
 * 1 <= dk, dv <= 128 (the tensor-core path needs dk = dv = 128 and bf16
 * q/k/v; every other size runs the CUDA-core path), 1 <= max_nodes <= 64,
 * T >= node_offset[R] rows in every per-node array, num_slots >= 1 blocks in
 * the state pool, R * H < 2^31 (request, head) pairs.
 *
 * Layouts (row-major, innermost index last; all device memory):
 *   node_offset  int32 [R+1], non-decreasing
 *   parent       int32 [T]        request-local parent index, -1 = hangs off S0
 *   q, k         bf16|f32 [T][H][dk]   (16-byte aligned base)
 *   v            bf16|f32 [T][H][dv]   (16-byte aligned base)
 *   alpha, beta  f32 [T][H]       decay gate and write strength, in (0,1)
 *   state        f32 [num_slots][H][dv][dk]  committed states S0 (row d of a
 *                                 head's state holds S0[d][0..dk-1]); 16-byte aligned;
 *                                 bf16, same shape, with TREEWY_FLAG_STATE_BF16
 *   state_slot   int32 [R]        pool slot of each request, in [0, num_slots)
 *   o            f32 [T][H][dv]   verify output o_n (16-byte aligned base)
 *   U            f32 [T][H][dv]   verify output u_n, commit input (16-byte
 *                                 aligned base; keep it
 *                                 alive from verify to commit: it replaces
 *                                 the per-node snapshots)
 *   gamma        f32 [T][H]       optional verify output gamma_n (may be NULL)
 *   status       int32 [R]        per-request error bits, OR-ed (see above)
 * The per-node arrays (parent, q, k, v, alpha, beta, o, U, gamma) may be
 * NULL when T = 0, a batch whose trees are all empty.
 */
typedef struct treewy_batch {
  int32_t R;
  int32_t H;
  int32_t dk;
  int32_t dv;
  int32_t max_nodes;
  int32_t qkv_dtype;
  int64_t T;
  int64_t num_slots;
  const int32_t* node_offset;
  const int32_t* parent;
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  void* state;                    /* f32, or bf16 with TREEWY_FLAG_STATE_BF16 */
  const int32_t* state_slot;
  float* o;
  float* U;
  float* gamma;
  int32_t* status;
  uint32_t flags;
  uint32_t reserved;
} treewy_batch;

/*
 * treewy_verify -- TreeWY verification of every draft node
 * (paper §3 "Verifying a draft", Eq. (2); review §3.2 Algorithm, steps 1-5).
 *
 * Reads node_offset, parent, q, k, v, alpha, beta, state (through
 * state_slot); writes o, U, gamma (if non-NULL) and ORs error bits into
 * status[r].  The outputs of a request with an error bit are left untouched.
 * The state is not modified.
 */
treewy_status treewy_verify(const treewy_batch* batch, cudaStream_t stream);

/*
 * treewy_commit -- reconstruct the accepted state in place
 * (paper §3 "Reconstruct on commit", Eq. (3); review §3.3, Eq. (6)).
 *
 * accepted: device int32 [R], request-local index of the accepted node, or -1
 * when no draft node is accepted (the state is then left untouched and not
 * read).  Reads node_offset, parent, alpha, k, U (from treewy_verify on the
 * same inputs) and state; overwrites state[state_slot[r]] with S_a.  q, v and
 * o are not read.  Requests with a bad tree or accepted index get status bits
 * OR-ed into status[r] and keep their state.  Requests must map to distinct
 * slots (two requests committing into one slot race).
 */
treewy_status treewy_commit(const treewy_batch* batch, const int32_t* accepted,
                            cudaStream_t stream);

/*
 * treewy_commit_verify -- the previous round's commit fused into this round's
 * verification (the deferred state write that the paper's §6 and the review's
 * §7(c)(3) point to: write the accepted state once, inside the next pass that
 * reads it).
 *
 * For every request r, state[state_slot[r]] holds S0 of the previous round;
 * `prev` describes that round (node_offset, parent, alpha, k and U from its
 * treewy_verify; q, v, o, beta are not read) and prev_accepted its accepted
 * nodes (device int32 [R], -1 = nothing accepted).  The kernel rebuilds
 * S_a = gamma_a S0 + sum_{i on path(a)} (gamma_a/gamma_i) u_i k_i^T on chip,
 * writes it back to the state block once, and verifies `next` from it: the
 * results equal treewy_commit(prev, prev_accepted) followed by
 * treewy_verify(next), with one state read per head instead of two.  (Shapes
 * other than dk = dv = 128 with bf16 q/k/v in both rounds, and a bf16 pool
 * whose next trees have at most 8 nodes while the previous ones have more
 * than 8, or 9 to 32 nodes while the previous ones have more than 16,
 * run as those two calls back to back on `stream`.)  A request with no node
 * in `next` still gets its commit.  prev and next must have the
 * same R, H, dk, dv, state pool pointer, num_slots, state_slot pointer and
 * TREEWY_FLAG_STATE_BF16.
 * Errors, as for the two calls made one after the other, with every status
 * bit going to next->status:
 *   - an error in the previous round (its tree, node range or accepted index)
 *     refuses that request's commit: its state is left unchanged, the bits of
 *     the reason are set together with TREEWY_STATUS_COMMIT_REFUSED, and `next`
 *     is still verified, from the unchanged state;
 *   - an error in `next` (its tree or node range) skips that request's
 *     verification (outputs untouched) but not its commit: S_a is written;
 *   - a state slot outside the pool refuses both (TREEWY_STATUS_BAD_SLOT |
 *     TREEWY_STATUS_COMMIT_REFUSED when a node was accepted).
 * So S_a was written for request r exactly when prev_accepted[r] >= 0 and
 * TREEWY_STATUS_COMMIT_REFUSED is clear in next->status[r].
 */
treewy_status treewy_commit_verify(const treewy_batch* prev, const int32_t* prev_accepted,
                                   const treewy_batch* next, cudaStream_t stream);

/*
 * treewy_storeall_verify -- the snapshot-per-node comparator ("storeall", the
 * full-state snapshotting of paper §2, approach (i)).
 *
 * Applies the gated delta rule node by node and writes every node's state to
 * snapshots, plus o (and U is not written).  snapshots: device f32
 * [T'][H][dv][dk] where T' = node_offset[R] - node_offset[0]: snapshot rows
 * are indexed relative to the batch's first node, so a caller can verify a
 * large batch in request chunks (pass node_offset + r0 and R_chunk) with
 * snapshot memory for one chunk only.  16-byte aligned.  status as in
 * treewy_verify.
 */
treewy_status treewy_storeall_verify(const treewy_batch* batch, float* snapshots,
                                     cudaStream_t stream);

/*
 * treewy_storeall_commit -- storeall rollback: copy the accepted node's
 * snapshot into state[state_slot[r]] (nothing for accepted = -1).
 * snapshots indexed as in treewy_storeall_verify for the same batch.
 */
treewy_status treewy_storeall_commit(const treewy_batch* batch, const float* snapshots,
                                     const int32_t* accepted, cudaStream_t stream);

/*
 * treewy_selftest_wait_timeout -- diagnostic of the kernels' bounded waits.
 *
 * Launches one thread that waits, with the same bounded wait every kernel
 * uses on its barriers, for a barrier phase that nothing completes, giving
 * up after limit_us microseconds (1 .. 10,000,000).  It then ORs
 * TREEWY_STATUS_TIMEOUT into status[0] and writes the measured wait in
 * nanoseconds to the two int32 words status[1] (low) and status[2] (high).
 * status: device int32 [3], caller-owned; the caller zeroes status[0].
 * Shows that a wait which never completes returns control, reports through
 * the status word and leaves the CUDA context usable.
 */
treewy_status treewy_selftest_wait_timeout(int32_t* status, uint32_t limit_us,
                                           cudaStream_t stream);

/*
 * One GDN layer's new tokens for a batch of sequences (treewy_extend).
 *
 * Sizes: R >= 0 sequences, H >= 1 value heads, Hk >= 1 key heads with H a
 * multiple of Hk (value head h reads q and k of head h / (H / Hk)),
 * 1 <= dk, dv <= 128, T >= seq_offset[R] token rows, max_len >= 0 a bound on
 * every sequence's number of new tokens that the host knows (it chooses the
 * kernel, one for the whole call: 1 where every sequence brings at most one
 * token), num_slots >= 1, R * H < 2^31.
 *
 * Layouts (device memory; innermost index last):
 *   seq_offset  int32 [R+1], non-decreasing: sequence r's tokens, in their
 *               order, are rows seq_offset[r] .. seq_offset[r+1]-1 (it may
 *               have none)
 *   q, k        bf16|f32, token t's row of [Hk][dk] at element t * q_stride
 *               (k_stride); strides 0 mean dense rows, others are at least
 *               Hk * dk (a slice of a fused projection)
 *   v           the same type, rows of [H][dv], stride v_stride
 *   alpha, beta f32 [T][H]: decay in [0, 1] and write strength
 *   state       the pool [num_slots][H][dv][dk] of treewy_batch: f32, or bf16
 *               with TREEWY_FLAG_STATE_BF16; 16-byte aligned
 *   state_slot  int32 [R], distinct (two sequences on one slot race)
 *   fresh       uint8 [R] or NULL: non-zero where the sequence starts from the
 *               zero state, which is then not read
 *   o           f32 or bf16 (o_dtype) [T][H][dv]
 *   status      int32 [R], bits OR-ed in
 * Everything but the state is aligned to its element size only; rows and bases that
 * are multiples of 16 bytes take the wide loads.  o and status overlap nothing
 * else.
 */
typedef struct treewy_seqs {
  int32_t R;
  int32_t H;
  int32_t Hk;
  int32_t dk;
  int32_t dv;
  int32_t max_len;
  int32_t qkv_dtype;
  int32_t o_dtype;
  int64_t T;
  int64_t num_slots;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  const int32_t* seq_offset;
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  void* state;
  const int32_t* state_slot;
  const uint8_t* fresh;
  void* o;
  int32_t* status;
  uint32_t flags;                 /* TREEWY_FLAG_FORCE_GENERIC, TREEWY_FLAG_STATE_BF16 */
  uint32_t reserved;
} treewy_seqs;

/*
 * treewy_extend -- the gated delta rule over every sequence's new tokens
 * (paper §1 Eq. (1)): from S = state[state_slot[r]] (zero where fresh),
 *   S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,  o_t = S_t q_t,
 * for the tokens of sequence r in order; o gets every o_t and the slot the
 * last state (rounded to nearest for a bf16 pool; S is f32 in between).  One
 * token per sequence is a decode step without a draft, many are a prompt or
 * a chunk of one.  A sequence without tokens keeps its state, or gets the
 * zero state where fresh.
 *
 * A token range outside [0, T) sets TREEWY_STATUS_BAD_TREE, a length that is
 * negative or above max_len TREEWY_STATUS_TOO_MANY_NODES, a slot outside the
 * pool TREEWY_STATUS_BAD_SLOT; that sequence's outputs and state stay as they
 * are.
 *
 * Long sequences of bf16 q, k and v with 16-byte rows run in chunks of 64
 * tokens on the tensor cores, f32 operands as bf16 terms.  For unit keys, the
 * state and f32 outputs are then within 2^-14 of their largest value where
 * 0 <= beta <= 1, and within 2^-11 where beta <= 2 and keys are much alike
 * (512 tokens at a cosine of 0.99 without decay; errors of independent keys
 * are 5e-6 in the norm); bf16 outputs are within four times that and their own
 * rounding.  Other calls run token by token in f32 (1e-7 to 1e-6), as all do
 * with TREEWY_FLAG_FORCE_GENERIC.  So do calls with f32 outputs over a bf16
 * pool: a difference that turns a rounding of the stored state shows in f32
 * outputs of later calls.  It does so whichever call stored the state, so a
 * sequence is as near as f32 sums only where all calls over it have f32
 * outputs or that flag.
 *
 * One kernel takes the whole call, and a single token in a call of prompts
 * costs it a chunk.  So a step that brings prompts and single tokens is two
 * calls over the same rows (seq_offset, state_slot, fresh and status from the
 * first sequence of each kind on, and each kind's max_len): a prompt of 2000
 * tokens with 255 single tokens of 32 heads takes 785 us in one call, 311 us in
 * two (bf16 pool: 629 and 245 us).
 *
 * In a chunk a NaN or an infinity among a token's inputs can reach the outputs
 * of that sequence and head from up to 63 tokens before it on.
 * TREEWY_STATUS_TIMEOUT: a wait of the kernel gave up; the sequence's outputs
 * are partly written and its state may be too.
 */
treewy_status treewy_extend(const treewy_seqs* seqs, cudaStream_t stream);

/* Norms of treewy_qk_norm. */
enum {
  TREEWY_NORM_L2 = 0,   /* x / sqrt(sum x^2 + eps) */
  TREEWY_NORM_RMS = 1   /* x / sqrt(mean x^2 + eps) */
};

/*
 * Queries and keys of T tokens for treewy_qk_norm.
 *
 * q (k): token t's row of [Hq][d] ([Hk][d]) at element t * q_stride
 * (k_stride), bf16 or f32; stride 0 means dense.  q_out, k_out: the same
 * type, dense rows of [Hq * q_repeat][d] ([Hk * k_repeat][d]): output heads
 * j * repeat .. j * repeat + repeat - 1 are head j, so that GDN layers whose
 * key heads are shared get the one row per value head that treewy_verify
 * reads.  q_out may be q itself where q_repeat is 1 and q is dense (k_out
 * likewise); other overlaps are not allowed.  Either side may be left out
 * (Hq = 0 or Hk = 0).  1 <= d <= 256.
 *   q_weight, k_weight  f32 [d] or NULL (ones)
 *   rope      f32 [rope_rows][rope_dims]: cosines of the rope_dims / 2 pairs,
 *             then their sines; rope_dims even, 0 .. d, 0 for no rotation
 *   position  int32 [T], rows of rope
 *   status    int32 [1]; TREEWY_STATUS_BAD_POSITION is OR-ed into it where a
 *             position is outside the table, and that token's outputs stay
 *             as they are.  May be NULL where rope_dims = 0.
 */
typedef struct treewy_qk {
  int64_t T;
  int32_t Hq;
  int32_t Hk;
  int32_t d;
  int32_t dtype;                  /* TREEWY_DTYPE_BF16 or TREEWY_DTYPE_F32 */
  int32_t norm;
  int32_t rope_dims;
  int32_t interleaved;            /* pairs (2i, 2i+1) instead of (i, i + rope_dims / 2) */
  int32_t q_repeat;
  int32_t k_repeat;
  float eps;
  float q_scale;                  /* factors of the normed rows, 1 for none */
  float k_scale;
  int64_t q_stride;
  int64_t k_stride;
  int64_t rope_rows;
  const void* q;
  const void* k;
  const float* q_weight;
  const float* k_weight;
  const float* rope;
  const int32_t* position;
  void* q_out;
  void* k_out;
  int32_t* status;
} treewy_qk;

/*
 * treewy_qk_norm -- every query and key head's norm, weight, scale and
 * position rotation in one pass, in f32 with one rounding at the end:
 *   y = scale w x / sqrt(sum or mean of x^2 + eps),
 *   (a, b) <- (a cos - b sin, b cos + a sin) for each rotated pair.
 */
treewy_status treewy_qk_norm(const treewy_qk* qk, cudaStream_t stream);

/*
 * Moves between slots of `layers` state pools for treewy_copy_slots: layer
 * l's pool starts at state + l * layer_stride bytes and holds num_slots
 * blocks of slot_bytes bytes.  src, dst: int32 [n] (device).  status: int32
 * [n], bits OR-ed in per move.
 */
typedef struct treewy_slots {
  int32_t n;
  int32_t layers;
  int64_t num_slots;
  int64_t slot_bytes;
  int64_t layer_stride;           /* bytes; 0: num_slots * slot_bytes */
  void* state;
  const int32_t* src;
  const int32_t* dst;
  int32_t* status;
} treewy_slots;

/*
 * treewy_copy_slots -- copies block src[i] to block dst[i] in every layer's
 * pool, byte for byte; src[i] = -1 fills block dst[i] with zeros (a request's
 * states forked to samples of it, live slots moved into holes, slots
 * cleared).  A source may serve several moves; a move with src[i] = dst[i]
 * does nothing and meets no other one.  Moves must not meet: where dst[i] is another
 * move's destination too, or src[i] another move's destination,
 * TREEWY_STATUS_SLOT_CLASH is set in status[i] and move i is not made.  An
 * index outside the pool sets TREEWY_STATUS_BAD_SLOT and the move is not
 * made (it still counts as a destination or source of its other index).
 */
treewy_status treewy_copy_slots(const treewy_slots* slots, cudaStream_t stream);

/*
 * One softmax layer's keys and values in 8 bits (treewy_attend, treewy_append):
 * a pool of pages of page_len tokens, e4m3 codes with an f32 scale for each
 * page and head, so that a key is k_scale times its code.
 *
 *   k, v        e4m3 [num_pages][Hkv][page_len][d], 16-byte aligned
 *   k_scale, v_scale  f32 [num_pages][Hkv], positive; treewy_append makes them
 *               powers of two, treewy_attend takes any in [2^-60, 2^60]
 *   page_table  int32 [R][max_pages]: token t of request r is row t % page_len
 *               of page page_table[r][t / page_len]; entries behind the
 *               request's tokens are not read
 *   length      int32 [R]: tokens in the cache
 * page_len is 16, 32, 64 or 128, 1 <= d <= 256, num_pages * Hkv < 2^31.  Full
 * pages may be shared by requests (a common prefix); a page that
 * treewy_append writes to belongs to one request and stands in its table once
 * (to fork a context whose last page is partly filled, copy that page first).
 * What a page holds behind its tokens may be anything.
 */
typedef struct treewy_cache {
  int32_t Hkv;
  int32_t d;
  int32_t page_len;
  int32_t max_pages;
  int64_t num_pages;
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  const int32_t* length;
} treewy_cache;

/*
 * Draft trees in front of a softmax layer (treewy_attend).
 *
 * Sizes: R >= 0 requests, Hq >= 1 query heads, a multiple of Hkv (query head
 * h reads key head h / (Hq / Hkv)), 1 <= max_nodes <= 64 a bound on every
 * request's nodes, max_context >= 0 a bound on every length (both known to the
 * host, which divides the work by them), T >= node_offset[R] rows.
 *   node_offset int32 [R+1], as in treewy_batch; a lone token is a tree of one
 *               node
 *   parent      int32 [T] as in treewy_batch (-1: hangs off the context), or
 *               NULL: every request's nodes are a chain
 *   q           bf16|f32, token t's row of [Hq][d] at element t * q_stride
 *   k, v        the same type, rows of [Hkv][d], the nodes' own keys and values
 *               (normed and rotated; they enter the cache by treewy_append).
 *               Strides 0 mean dense rows
 *   o           bf16|f32 (o_dtype) [T][Hq][d]
 *   status      int32 [R], bits OR-ed in
 *   scale       factor of the scores, positive (1/sqrt(d))
 *   workspace   workspace_bytes of device memory, 16-byte aligned, at least
 *               what treewy_attend_workspace says; one call at a time uses it.
 *               It needs no contents before a call and keeps none after it.
 * Everything but the pages and the workspace is aligned to its element size;
 * o and status overlap nothing else.
 */
typedef struct treewy_attn {
  int32_t R;
  int32_t Hq;
  int32_t max_nodes;
  int32_t max_context;
  int32_t qkv_dtype;
  int32_t o_dtype;
  int64_t T;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  const int32_t* node_offset;
  const int32_t* parent;
  const void* q;
  const void* k;
  const void* v;
  void* o;
  int32_t* status;
  void* workspace;
  uint64_t workspace_bytes;
  float scale;
  uint32_t flags;                 /* TREEWY_FLAG_FORCE_GENERIC */
  treewy_cache cache;
} treewy_attn;

/*
 * treewy_attend -- softmax attention of every draft node over its request's
 * context and its own path in the draft: for node n,
 *   s_j = scale q_n . k_j,  o_n = sum_j e^{s_j} v_j / sum_j e^{s_j},
 * j over the length[r] tokens in the cache, n's ancestors and n itself.  So no
 * node is without a key.  The cache is not changed: as with treewy_verify and
 * treewy_commit, what is accepted goes in afterwards.
 *
 * A node range outside [0, T) or a bad parent sets TREEWY_STATUS_BAD_TREE,
 * more than max_nodes nodes TREEWY_STATUS_TOO_MANY_NODES, a page or length that
 * does not hold TREEWY_STATUS_BAD_PAGE; that request's outputs stay as they are
 * (with TREEWY_STATUS_TIMEOUT, some may be written).
 *
 * bf16 rows with bf16 outputs and d a multiple of 16 run on the tensor cores in
 * 8-bit products, every f32 or bf16 operand as two 8-bit terms: a query, key or
 * value of the draft is within 2^-17 of its row's largest (or 2^-117), a weight
 * of the softmax within 2^-8 of itself or 2^-17 of its row's largest (2^-21
 * where that stands out from the others, or with at most 16 rows: nodes times
 * query heads of a key head).  Other calls run in f32.
 *
 * A NaN (or an infinity, which counts as one) in a key reaches every node that
 * sees it, in a value every such node's column, in a query its own row.  Where a
 * score overflows f32, the node's outputs are NaN (on the tensor cores one that
 * overflows below counts for nothing).
 */
treewy_status treewy_attend(const treewy_attn* attn, cudaStream_t stream);

/* Bytes of workspace that treewy_attend needs for arguments of these sizes
   (R, T, Hq, max_nodes, max_context, the types, flags and the cache's sizes are
   read, no pointers): on a card of any number of SMs, and for any contents. */
treewy_status treewy_attend_workspace(const treewy_attn* attn, uint64_t* bytes);

/*
 * New keys and values for a cache (treewy_append).
 *
 * node_offset, T, strides: as in treewy_attn.  accepted NULL: every row of
 * request r, in order, goes behind its length[r] tokens.  accepted int32 [R]:
 * the rows on the path from the root to node accepted[r] do (-1: none), for
 * trees of at most 64 nodes (parent NULL: chains).  max_new: a bound on every
 * request's rows.  k, v: bf16|f32 (kv_dtype) rows of [Hkv][d].
 *   new_length  int32 [R] or NULL: length[r] and the rows taken.  It is not
 *               cache.length itself, which all layers of a step read.
 */
typedef struct treewy_append_args {
  int32_t R;
  int32_t max_new;
  int32_t kv_dtype;
  uint32_t reserved;
  int64_t T;
  int64_t k_stride;
  int64_t v_stride;
  const int32_t* node_offset;
  const int32_t* parent;
  const int32_t* accepted;
  const void* k;
  const void* v;
  int32_t* new_length;
  int32_t* status;
  treewy_cache cache;
} treewy_append_args;

/*
 * treewy_append -- rows into their pages, rounded to e4m3 in units of the
 * page's scale (for each head; keys and values apart).  Values up to 2^68 give
 * scales that treewy_attend takes.
 *
 * A page's scale is the least power of two, 2^-40 at least, that brings what is
 * written to it within 448, e4m3's largest value.  Where a page has tokens
 * already, its scale only grows: then the codes of those tokens are divided by
 * the same power of two, which is exact but for codes that leave e4m3's normal
 * range.  A NaN or an infinity is stored as NaN and does not count for the
 * scale.  Rows of a page behind its tokens stay as they are.
 *
 * A node range outside [0, T) or a bad parent sets TREEWY_STATUS_BAD_TREE,
 * more than max_new rows TREEWY_STATUS_TOO_MANY_NODES, accepted[r] outside
 * [-1, N_r) TREEWY_STATUS_BAD_ACCEPTED, a length that does not fit the pages or
 * a page outside the pool TREEWY_STATUS_BAD_PAGE; nothing of that request is
 * written.
 */
treewy_status treewy_append(const treewy_append_args* args, cudaStream_t stream);

/*
 * Rows for treewy_add_norm: T rows of n, 1 <= n <= 32768.
 *   x             bf16|f32 (x_dtype), row t at element t * x_stride (0: dense)
 *   residual      bf16|f32 (residual_dtype) or NULL, stride residual_stride
 *   residual_out  the same type, dense rows, needed with a residual; it may be
 *                 residual itself where that is dense
 *   weight        f32 [n] or NULL (ones)
 *   y             x's type, dense rows, or NULL; it may be x itself where that
 *                 is dense
 *   y8            e4m3, dense rows, or NULL
 *   y8_scale      f32 [T][ceil(n / group)], needed with y8; group is 32, 64 or
 *                 128 columns, or 0: one scale for a row
 * Other overlaps are not allowed; everything is aligned to its element size.
 */
typedef struct treewy_norm {
  int64_t T;
  int64_t x_stride;
  int64_t residual_stride;
  int32_t n;
  int32_t x_dtype;
  int32_t residual_dtype;
  int32_t group;
  float eps;
  uint32_t reserved;
  const void* x;
  const void* residual;
  void* residual_out;
  const float* weight;
  void* y;
  void* y8;
  float* y8_scale;
} treewy_norm;

/*
 * treewy_add_norm -- the residual's addition and the RMS norm in one pass:
 *   z = x + residual,  y = w z / sqrt(mean of z^2 + eps),
 * in f32 (so a row whose squares pass f32 is normed to zeros); residual_out gets
 * z, y and y8 the norm of z before its rounding.  A group's scale is its largest
 * |y| / 448, 2^-126 at least (1 where all are 0), and y8 is y times 1 / scale in
 * f32 rounded to e4m3: where y / scale is within 2^-22 of the middle between two
 * codes, either one.  NaN stays NaN and does not count for the scale; an infinite
 * y makes the scale infinite, its own code NaN and the group's others 0.
 */
treewy_status treewy_add_norm(const treewy_norm* norm, cudaStream_t stream);

/* Message for the last non-OK return on the calling host thread ("" if none). */
const char* treewy_last_error(void);

/* Library version string. */
const char* treewy_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TREEWY_H */
