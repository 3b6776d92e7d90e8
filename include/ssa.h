/*
 * ssa.h -- C ABI of libssa: DAM structured sparse attention on one B200 (sm_100a).
 *
 * The method is the Dynamic Attention Mask of the DAM review page ("DAM: Dynamic
 * Attention Mask for Long-Context Large Language Model Inference Acceleration",
 * pith review of arXiv 2506.11104):
 *   stage one  ("What carries the argument"): averaged L x L attention maps ->
 *              Box-Cox (lambda) -> threshold tau -> binary true mask M -> score every
 *              diagonal (j = i - r) and vertical (j = c, i >= c) candidate by
 *              gamma_k = sum(M P_k) / sum(P_k) -> keep gamma_k >= mu;
 *   stage two  ("What carries the argument"; "Circularity Check", steps 1 and 2;
 *              Referee Report summary): the kept patterns, pasted over S x S, form
 *              the extended mask applied to QK^T / sqrt(d_k) before the softmax.
 *
 * Conventions shared by every call
 *   - Every call returns an int status (SSA_OK or a negative SSA_ERR_* code) and
 *     records a message retrievable with ssa_last_error() (thread-local).
 *   - The caller owns all memory.  Every pointer argument named as "device" must
 *     point to CUDA device memory of the current device; "host" pointers to host
 *     memory.  The library allocates and frees nothing and never synchronises the
 *     stream, except where a call says so.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream).
 *     All work of a call is enqueued on it, in order.
 *   - `dev_status` (device, one int32, may be NULL) receives faults detected on the
 *     GPU: the first non-zero SSA_ERR_* code written by any kernel stays.  The caller
 *     zeroes it and reads it after synchronising.  Kernels never trap: on a bad index
 *     or an expired bounded wait they record the code and return.
 *   - bf16 tensors are passed as raw 16-bit storage (uint16_t / void*).
 */
#ifndef SSA_H
#define SSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define SSA_API __attribute__((visibility("default")))
#else
#define SSA_API
#endif

#define SSA_OK 0
#define SSA_ERR_INVALID (-1)     /* null pointer, bad size, unsorted/duplicate/negative list, bad map entry */
#define SSA_ERR_UNSUPPORTED (-2) /* head dim not 64/128, capture L > 1024, Case-2 plan given to decoding,
                                    an unknown cache format, a kernel build or device ordinal the
                                    library cannot use */
#define SSA_ERR_CAPACITY (-3)    /* caller buffer or workspace too small */
#define SSA_ERR_CUDA (-4)        /* a CUDA runtime/driver call failed */
#define SSA_ERR_TIMEOUT (-5)     /* a bounded on-device wait expired */

/* Tile edge of the query blocks and key tiles used by the plan and the kernels. */
#define SSA_BLOCK 128

/* ------------------------------------------------------------------------------ */
/* Stage one: averaged attention maps                                              */
/* ------------------------------------------------------------------------------ */

#define SSA_MAPS_MAX_B 32   /* samples averaged per call */
#define SSA_MAPS_MAX_L 4096

/*
 * sparse_attn_maps -- the averaged attention maps stage one starts from ("What carries
 * the argument": maps averaged over a calibration corpus; "Assumptions & free
 * parameters": capture length L = 512), produced on the GPU from B samples of each
 * map's query and key rows:
 *   maps[m][i][j] = (1/B) sum_b softmax_j( scale * Q[m][b][i] . K[m][b][j] )   j <= i
 *   maps[m][i][j] = 0                                                          j > i
 * (causal row softmax per sample, then the mean over the samples), in the layout
 * sparse_pattern_capture reads.  Arithmetic: bf16 inputs, fp32 logits (tensor cores),
 * fp32 softmax with hardware 2^x, fp32 mean; each row sums to 1 up to fp32 rounding.
 *
 *   Q, K     device, bf16 [n_maps][B][L][d] contiguous (sample b of map m at
 *            (m * B + b) * L * d), 16-byte aligned
 *   n_maps   >= 1 with n_maps * L < 2^31 and n_maps * B < 2^30;  B in [1, SSA_MAPS_MAX_B];
 *            L a multiple of 128 in [128, SSA_MAPS_MAX_L]
 *   d        64 or 128 (else SSA_ERR_UNSUPPORTED)
 *   scale    > 0, usually 1 / sqrt(d)
 *   maps     device, float32 [n_maps][L][L] row-major, 16-byte aligned; every entry
 *            is written
 * Errors: SSA_ERR_INVALID for a null or misaligned pointer or a size out of range; an
 * expired bounded wait sets SSA_ERR_TIMEOUT in dev_status (maps then unspecified).
 * For B larger than SSA_MAPS_MAX_B, average the maps of several calls weighted by
 * their sample counts.
 */
SSA_API int sparse_attn_maps(const void *Q, const void *K, int n_maps, int B, int L, int d, float scale,
                             float *maps, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------ */
/* Stage one: pattern capture                                                      */
/* ------------------------------------------------------------------------------ */

/* Workspace bytes sparse_pattern_capture needs for n_maps maps of size L x L. */
SSA_API size_t sparse_pattern_capture_ws_bytes(int n_maps, int L);

/*
 * sparse_pattern_capture -- stage one of DAM ("What carries the argument"; lambda,
 * tau, mu from "Assumptions & free parameters"; eps from Referee Report minor
 * comment 1).
 *
 * For every map m and row i (causal entries j <= i only):
 *   y_j = ((x_j + eps)^lambda - 1) / lambda                (Box-Cox)
 *   t_j = (y_j - y_min) / (y_max - y_min)  (row min/max; t = 1 on a constant row)
 *   M[i][j] = t_j >= tau
 * then gamma_diag[r] = #{i >= r : M[i][i-r]} / (L - r), gamma_vert[c] =
 * #{i >= c : M[i][c]} / (L - c), both in fp64, and r (resp. c) is kept iff
 * gamma >= mu.  At lambda 0.5 and 1 every threshold decision is made with correctly
 * rounded fp64 arithmetic in the stated order, so the kept lists are exactly
 * reproducible.  Other lambdas (0 = log) go through fp64 pow / log, which are not
 * correctly rounded: an entry whose t lies within a few units in the last place of
 * tau may be decided differently by another implementation.
 *
 *   maps         device, float32 [n_maps][L][L] row-major, already averaged over the
 *                calibration batches; causal entries must be finite and >= 0
 *                (entries j > i are ignored)
 *   n_maps       >= 1;  L in [1, 1024]
 *   lambda       in [0, 64] (else SSA_ERR_INVALID); tau, mu in fp64; eps >= 0
 *   diag_ptr     device int32 [n_maps + 1]   CSR row pointers of the kept diagonals
 *   diag_offsets device int32 [n_maps * L]   kept r, ascending within each map
 *   vert_ptr     device int32 [n_maps + 1]
 *   vert_cols    device int32 [n_maps * L]   kept c, ascending within each map
 *   ws           device workspace of at least sparse_pattern_capture_ws_bytes()
 * A negative or non-finite map entry sets SSA_ERR_INVALID in dev_status; the lists
 * are then unspecified.  When maps is 16-byte aligned and L a multiple of 4, rows are
 * staged into shared memory by bulk copies whose waits are bounded
 * (ssa_set_wait_limit_ns): an expired wait sets SSA_ERR_TIMEOUT in dev_status, the
 * kernel waits (again bounded) for its copies in flight and the lists are unspecified.
 */
SSA_API int sparse_pattern_capture(const float *maps, int n_maps, int L, double lambda, double tau,
                           double mu, double eps, int32_t *diag_ptr, int32_t *diag_offsets,
                           int32_t *vert_ptr, int32_t *vert_cols, void *ws, size_t ws_bytes,
                           int32_t *dev_status, void *stream);

/* Scalings of the Box-Cox output to [0, 1] before tau (the page leaves it unstated). */
#define SSA_SCALE_ROW 0 /* min and max over each row's causal entries (the default reading) */
#define SSA_SCALE_MAP 1 /* min and max over all causal entries of the map */

/*
 * sparse_pattern_capture_ex -- sparse_pattern_capture with the two optional readings
 * and outputs of stage one:
 *   scaling    SSA_SCALE_ROW (as sparse_pattern_capture) or SSA_SCALE_MAP: every row
 *              of a map uses the map's min and max (a constant map has t = 1); this
 *              reading reads the maps twice (a min/max pass, then the decisions)
 *   true_mask  null, or device uint32 [n_maps][L][ceil(L/32)], 4-byte aligned: the
 *              binary true mask M itself, bit (j % 32) of word j / 32 of row i set iff
 *              j <= i and M[i][j] (the input of the Case-2 extension,
 *              sparse_pattern_extend_case2)
 * All other arguments, the workspace and the errors are those of
 * sparse_pattern_capture; a scaling other than the two is SSA_ERR_INVALID.
 */
SSA_API int sparse_pattern_capture_ex(const float *maps, int n_maps, int L, double lambda, double tau,
                                      double mu, double eps, int scaling, int32_t *diag_ptr,
                                      int32_t *diag_offsets, int32_t *vert_ptr, int32_t *vert_cols,
                                      uint32_t *true_mask, void *ws, size_t ws_bytes,
                                      int32_t *dev_status, void *stream);

/* Size of the fixed device scratch of sparse_pattern_capture_noalloc (8 MiB). */
#define SSA_CAPTURE_NOALLOC_SCRATCH_BYTES (8u << 20)

/*
 * sparse_pattern_capture_noalloc -- sparse_pattern_capture without a workspace
 * argument.  The paper has no counterpart: this is a deployment variant.
 *
 * For callers that cannot allocate device memory: a plugin host that only hands the
 * library its input and output buffers and has no allocator to lend, or a serving
 * process that must not call cudaMalloc/cudaFree after start-up because those calls
 * can synchronise the device and stall every other stream.  The call itself allocates
 * nothing: its scratch is a fixed SSA_CAPTURE_NOALLOC_SCRATCH_BYTES device array
 * inside the library, held by every GPU that loads the library until the process
 * exits.  Arguments, outputs and results are those of sparse_pattern_capture; the
 * caller still provides maps, the four output lists and dev_status.
 *
 *   - Sizes whose scratch (sparse_pattern_capture_ws_bytes(n_maps, L)) exceeds the
 *     fixed size are rejected with SSA_ERR_CAPACITY before any device work
 *     (L = 512 allows up to 1023 maps).
 *   - The first call on each device looks up the array's device address with that
 *     device current and keeps it for the life of the process; make that first call
 *     before any stream capture begins.  A device reset (cudaDeviceReset, or anything
 *     else that tears down the primary context) invalidates the kept address: do not
 *     call this entry point again in a process that has reset the device.
 *   - Every call shares the one array per device and clears what must start at zero
 *     itself; calls that overlap on the GPU (different streams or host threads) race
 *     on it and must be serialised by the caller.
 */
SSA_API int sparse_pattern_capture_noalloc(const float *maps, int n_maps, int L, double lambda,
                                           double tau, double mu, double eps, int32_t *diag_ptr,
                                           int32_t *diag_offsets, int32_t *vert_ptr,
                                           int32_t *vert_cols, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------ */
/* Stage two: extension to S and the tile plan                                     */
/* ------------------------------------------------------------------------------ */

/* Sizes of a plan, filled by the sizing pass of sparse_pattern_extend. */
typedef struct ssa_plan_sizes {
    int32_t n_heads;
    int32_t S;
    int32_t nqb;       /* ceil(S / 128) */
    int32_t n_diag;    /* total extended diagonals over all heads */
    int32_t n_vert;    /* total extended columns over all heads */
    int32_t max_vert;  /* max over heads of the extended column count */
    int64_t n_tiles;   /* total listed band tiles */
    int32_t bitmap_slots; /* Case-2 plans: element-bitmap slots per head (0 otherwise) */
} ssa_plan_sizes;

/*
 * A compiled plan.  The struct itself is host memory; every pointer in it is a
 * device buffer owned by the caller and sized from ssa_plan_sizes:
 *   ext_diag_ptr [n_heads+1], ext_diag_offsets [max(n_diag,1)],
 *   ext_vert_ptr [n_heads+1], ext_vert_cols [max(n_vert,1)],
 *   tile_ptr [n_heads*nqb + 1], tile_key0 [max(n_tiles,1)],
 *   tile_dmask [max(n_tiles,1)][4] (uint64), tile_cmask [max(n_tiles,1)][2] (uint64),
 *   tile_flags [max(n_tiles,1)], stripe_cnt [n_heads*nqb].
 * Tile semantics, for head h and query block qb (rows lo = 128qb .. hi = 128qb+127):
 *   needed keys: j in [0, hi] such that some extended diagonal r has lo-j <= r <= hi-j
 *   (all 128 rows count, even in a ragged last block); the band tiles are key windows
 *   key0 .. key0+127, chosen greedily: the first starts at the smallest needed key,
 *   each next one at the smallest needed key >= previous key0 + 128 (so a band whose
 *   keys do not start at a multiple of 128 still takes ceil(width / 128) windows);
 *   dmask bit t (0..254) set  iff  r = 128qb - key0 + t - 127 is an extended diagonal
 *   cmask bit jl (0..127) set iff  column key0 + jl is an extended column
 *   a window is listed, in ascending key0, iff some (i, j) in it has i < S,
 *   i - j a diagonal and j not a column; tile_flags bit 0 (FULL) iff 128(qb+1) <= S,
 *   all 255 dmask bits set and cmask == 0;
 *   stripe_cnt[h*nqb+qb] = #{extended columns c <= min(S-1, 128qb+127)}.
 * The windows are disjoint and cover every needed key, and columns are owned by the
 * stripe phase only, so each retained pair is used once.
 */
typedef struct ssa_plan {
    int32_t n_heads;
    int32_t S;
    int32_t nqb;
    int32_t max_vert;
    int64_t n_tiles; /* capacity of the tile arrays (from ssa_plan_sizes) */
    int32_t *ext_diag_ptr;
    int32_t *ext_diag_offsets;
    int32_t *ext_vert_ptr;
    int32_t *ext_vert_cols;
    int32_t *tile_ptr;
    int32_t *tile_key0;
    uint64_t *tile_dmask;
    uint64_t *tile_cmask;
    uint32_t *tile_flags;
    int32_t *stripe_cnt;
    /* Case-2 plans only (sparse_pattern_extend_case2; zero / NULL otherwise): */
    int32_t bitmap_slots; /* from ssa_plan_sizes */
    uint64_t *tile_bits;  /* [n_heads * bitmap_slots][128][2] (uint64), 16-byte aligned */
    /* Capacities of ext_diag_offsets and ext_vert_cols (n_diag, n_vert from
     * ssa_plan_sizes).  A fill pass whose extended lists need more (in total, or more
     * than max_vert columns for one head) changes nothing in the plan and reports
     * SSA_ERR_CAPACITY in dev_status; the tile arrays are checked against n_tiles the
     * same way. */
    int32_t n_diag;
    int32_t n_vert;
} ssa_plan;

/* Workspace bytes of either pass of sparse_pattern_extend (about 4 * n_heads * S for
 * the per-diagonal run starts, plus small per-block counters). */
SSA_API size_t sparse_pattern_extend_ws_bytes(int n_heads, int S);

/*
 * sparse_pattern_extend -- stage two of DAM ("What carries the argument": the kept
 * patterns are pasted into an S x S mask; "Circularity Check" step 1: that mask is
 * the union of the matched patterns).  The extended lists keep every diagonal r < S
 * and column c < S of each head; the plan then lists, per query block, the key tiles
 * the band touches.
 *
 *   n_heads, S   >= 1
 *   diag_ptr, diag_offsets, vert_ptr, vert_cols
 *                device CSR lists per head (e.g. the output of capture); each list
 *                strictly ascending and >= 0, else SSA_ERR_INVALID
 *   sizes        host, always filled when plan == NULL (sizing pass)
 *   plan         NULL: sizing pass -- enqueues the counting kernels, copies the
 *                totals to the host and SYNCHRONISES `stream`; returns
 *                SSA_ERR_INVALID if a list is malformed, SSA_ERR_CAPACITY if the plan
 *                would hold more than INT32_MAX tiles (tile_ptr is int32).
 *                non-NULL: fill pass -- writes every plan array (no synchronisation);
 *                the new lists and tiles are counted in the workspace first, and only
 *                when they fit the plan's capacities (n_diag, n_vert, max_vert,
 *                n_tiles) is the plan written; otherwise it keeps its previous content
 *                and SSA_ERR_CAPACITY goes to dev_status.  plan->n_heads/S/nqb must
 *                match the call.
 *   ws           device workspace of at least sparse_pattern_extend_ws_bytes()
 */
SSA_API int sparse_pattern_extend(int n_heads, const int32_t *diag_ptr, const int32_t *diag_offsets,
                          const int32_t *vert_ptr, const int32_t *vert_cols, int S,
                          ssa_plan_sizes *sizes, const ssa_plan *plan, void *ws, size_t ws_bytes,
                          int32_t *dev_status, void *stream);

/*
 * sparse_pattern_extend_case2 -- the Case-2 reading of the extension (DAM review page,
 * Referee Report major comment 2: the patterns are pasted beyond the first L tokens):
 * the captured L x L true mask of each head is kept verbatim in the first block, the
 * union of the kept patterns everywhere else.  Cell (i, j), j <= i < S, is retained iff
 *   i < L:  bit j of row i of true_mask[h]     (the patterns play no part there)
 *   i >= L: i - j is a kept diagonal or j a kept column (as sparse_pattern_extend).
 * The paper has no tile plan; this is the library's layout: every query block holding
 * a row below min(L, S) is covered by element-bitmap tiles, one per key block kb = 0..qb
 * (key0 = 128 kb), listed when any of its cells is set, with tile_flags bit 1 (BITMAP),
 * the bitmap's slot h * bitmap_slots + qb (qb + 1) / 2 + kb in tile_dmask word 0, and
 * no stripe tiles (stripe_cnt 0); plan->tile_bits[slot][il][w] holds the cells of row il,
 * key column jl at bit jl % 64 of word jl / 64.  The other query blocks have the plan of
 * sparse_pattern_extend.
 *
 *   true_mask  device uint32 [n_heads][L][ceil(L/32)], 4-byte aligned, bit j % 32 of
 *              word j / 32 of row i = M[i][j] (sparse_pattern_capture_ex writes it;
 *              bits above the diagonal are ignored)
 *   L          capture length, [1, 1024]
 * Everything else as sparse_pattern_extend; the sizing pass also sets
 * sizes->bitmap_slots, and the fill pass needs plan->bitmap_slots equal to it and
 * plan->tile_bits (16-byte aligned) of n_heads * bitmap_slots * 128 * 2 uint64.
 * sparse_attn_fwd takes the plan as it is; sparse_attn_decode rejects it
 * (SSA_ERR_UNSUPPORTED: decoding follows the first reading only).
 */
SSA_API int sparse_pattern_extend_case2(int n_heads, const int32_t *diag_ptr, const int32_t *diag_offsets,
                                        const int32_t *vert_ptr, const int32_t *vert_cols,
                                        const uint32_t *true_mask, int L, int S, ssa_plan_sizes *sizes,
                                        const ssa_plan *plan, void *ws, size_t ws_bytes, int32_t *dev_status,
                                        void *stream);

/* ------------------------------------------------------------------------------ */
/* Attention forward                                                               */
/* ------------------------------------------------------------------------------ */

/* Workspace bytes of sparse_attn_fwd: a 256-byte work counter followed by the
 * gathered stripe keys and values. */
SSA_API size_t sparse_attn_fwd_ws_bytes(int n_heads, int max_vert, int d);

/*
 * sparse_attn_fwd -- causal prefill attention restricted to the extended mask
 * (Referee Report summary and "Circularity Check" step 2: the mask is applied to
 * QK^T / sqrt(d_k) before the softmax; "What carries the argument": only the
 * retained connections are computed).  For head h, KV head g = kv_map[h] (or
 * h / (H_q/H_kv) when kv_map is NULL) and query i < S, with retained keys
 * J_i = {i - r : r in D_h, r <= i} U {c in C_h : c <= i}:
 *   O[h][i]   = sum_{j in J_i} softmax_j(scale * q_i . k_j) v_j
 *   LSE[h][i] = log sum_{j in J_i} exp(scale * q_i . k_j)     (natural log)
 * An empty J_i gives O = 0 and LSE = -inf.  bf16 inputs, fp32 accumulation, bf16 O.
 *
 *   Q, O         device bf16 [H_q][S][d], contiguous
 *   K, V         device bf16 [H_kv][S][d], contiguous
 *   H_q, H_kv    >= 1; H_q % H_kv == 0 when kv_map is NULL
 *   S            must equal plan->S;  d in {64, 128} (else SSA_ERR_UNSUPPORTED)
 *   plan         host struct of device arrays from sparse_pattern_extend, n_heads == H_q
 *   kv_map       device int32 [H_q] or NULL; entries outside [0, H_kv) set
 *                SSA_ERR_INVALID in dev_status
 *   scale        softmax scale (1/sqrt(d) for the paper's formula)
 *   LSE          device float32 [H_q][S]
 *   ws           device workspace of at least sparse_attn_fwd_ws_bytes(H_q, plan->max_vert, d);
 *                all base pointers must be 16-byte aligned
 */
SSA_API int sparse_attn_fwd(const void *Q, const void *K, const void *V, int H_q, int H_kv, int S, int d,
                    const ssa_plan *plan, const int32_t *kv_map, float scale, void *O, float *LSE,
                    void *ws, size_t ws_bytes, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------ */
/* Decoding step                                                                   */
/* ------------------------------------------------------------------------------ */

/* Workspace bytes of sparse_attn_decode: the per-split partial results
 * ((2 + d) floats per split, 1 to 16 splits per sequence and head). */
SSA_API size_t sparse_attn_decode_ws_bytes(int B, int H_q, int d);

/*
 * sparse_attn_decode -- one decoding step over the same extended mask: the new query
 * of sequence b sits at position pos[b] and attends to row pos[b] of the mask ("What
 * carries the argument": the kept patterns are pasted over the whole S x S square;
 * Referee Report summary: the mask is applied to the scaled logits before the
 * softmax), i.e. for head h with KV head g:
 *   J = {pos - r : r an extended diagonal, r <= pos} U {c an extended column, c <= pos}
 *   O[b][h]   = sum_{j in J} softmax_j(scale * q . K[b][g][j]) V[b][g][j]
 *   LSE[b][h] = log sum_{j in J} exp(scale * q . K[b][g][j])      (natural log)
 * which is row pos[b] of sparse_attn_fwd over the same cache.  An empty J gives O = 0
 * and LSE = -inf.  bf16 inputs, fp32 accumulation, bf16 O.  Bound by the HBM traffic
 * of the gathered key and value rows.
 *
 *   Q, O         device bf16 [B][H_q][d], contiguous
 *   K, V         device bf16 [B][H_kv][S_cache][d]: the key/value cache of each sequence
 *   B, H_q, H_kv >= 1 (B, H_q <= 65535); H_q % H_kv == 0 when kv_map is NULL
 *   S_cache      must equal plan->S;  d in {64, 128} (else SSA_ERR_UNSUPPORTED)
 *   pos          device int32 [B], 0 <= pos[b] < S_cache; a position outside that range
 *                (or a kv_map entry outside [0, H_kv)) sets SSA_ERR_INVALID in
 *                dev_status and gives that sequence O = 0, LSE = -inf
 *   plan         from sparse_pattern_extend with S = S_cache and n_heads = H_q (only its
 *                extended lists are read)
 *   LSE          device float32 [B][H_q]
 *   ws           device workspace of at least sparse_attn_decode_ws_bytes(B, H_q, d);
 *                Q, K, V, O and ws 16-byte aligned
 */
SSA_API int sparse_attn_decode(const void *Q, const void *K, const void *V, int B, int H_q, int H_kv,
                               int S_cache, int d, const int32_t *pos, const ssa_plan *plan,
                               const int32_t *kv_map, float scale, void *O, float *LSE, void *ws,
                               size_t ws_bytes, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------ */
/* Key/value cache: append (norm, rotation, quantisation) and read back             */
/* ------------------------------------------------------------------------------ */

/* Cache formats.  The 8-bit and 4-bit ones hold groups of SSA_KV_GROUP consecutive
 * elements of a row with one scale byte E: the value is code * 2^(E - 127).  A scale is
 * a power of two, so scaling rounds nothing: a stored value is the nearest code (ties to
 * even) of y / 2^e, where e is the smallest exponent in range with max|y| <= M * 2^e
 * (M = 448 or 6, the largest code), and it is a bf16 number exactly.  e lies in
 * [-111, 7] (e4m3) or [-111, 13] (e2m1), E = e + 127: larger values saturate at
 * 448 * 2^7 = 57344 or 6 * 2^13 = 49152.  A group that holds a NaN or an infinity is
 * stored as codes 0 with E = 255 and reads back as NaN.  A cache made elsewhere holds
 * E from 16 to 134 (e4m3) or 140 (e2m1), 255 with codes 0, or 0 with codes 0 (a row never
 * written).  An E above that in a row that a call reads sets SSA_ERR_INVALID in dev_status, and
 * the row's values are unspecified; values of one from 1 to 15 may round to zero. */
#define SSA_KV_BF16 0 /* bf16 rows, no scales */
#define SSA_KV_E4M3 1 /* 8 bits: sign, 4 exponent, 3 mantissa bits, one byte an element */
#define SSA_KV_E2M1 2 /* 4 bits: sign, 2 exponent, 1 mantissa bit, two to a byte, even element low */
#define SSA_KV_GROUP 32

/*
 * A key/value cache.  The struct itself is host memory; its pointers are device buffers
 * owned by the caller, 16-byte aligned, contiguous:
 *   k, v              [B][H_kv][S] rows of d bf16 values, d e4m3 codes or d/2 bytes of
 *                     e2m1 codes
 *   k_scale, v_scale  [B][H_kv][S][d / SSA_KV_GROUP] scale bytes E (NULL for SSA_KV_BF16)
 * d is 64 or 128.
 */
typedef struct ssa_kv_cache {
    int32_t format; /* SSA_KV_* */
    int32_t B;
    int32_t H_kv;
    int32_t S; /* rows per sequence and head */
    int32_t d;
    void *k;
    void *v;
    uint8_t *k_scale;
    uint8_t *v_scale;
} ssa_kv_cache;

/* A bf16 array of [tokens][heads][d] rows: row (t, h) starts at element
 * t * token_stride + h * head_stride, its d elements are contiguous.  The base is 16-byte
 * aligned and the strides are non-negative multiples of 8 elements.  A projection's output
 * (token-major), a slice of a joint projection, and the head-major [heads][tokens][d] that
 * sparse_attn_fwd takes are all such views. */
typedef struct ssa_rows {
    void *ptr; /* NULL: absent */
    int64_t token_stride;
    int64_t head_stride;
} ssa_rows;

/*
 * Arguments of sparse_kv_append.  Sequence b owns the tokens t in
 * [tok_ptr[b], tok_ptr[b+1]); token t goes to its cache row row0[b] + (t - tok_ptr[b]),
 * so no two tokens share a row.  Tokens before tok_ptr[0] and from tok_ptr[B] on are
 * padding: nothing of theirs is used or written.
 */
typedef struct ssa_kv_append_args {
    int32_t n_tokens; /* tokens the views hold; tok_ptr[B] <= n_tokens */
    int32_t H_q;      /* query heads; 0 with q and q_out absent */
    ssa_rows q, k, v; /* projections; k and v have the cache's H_kv heads */
    ssa_rows q_out;   /* normalised and rotated queries (may be q itself) */
    ssa_rows k_out, v_out; /* optional: the values the cache now stands for, as bf16 (exact);
                              both or neither, may be k and v themselves */
    const int32_t *tok_ptr; /* device [B + 1], ascending, >= 0 */
    const int32_t *row0;    /* device [B], >= 0 */
    const int32_t *pos;     /* device [n_tokens] rotation position >= 0 of each token, or NULL:
                               its cache row (a drafted token sits at another position) */
    const double *freqs;    /* device [d / 2] radians per position, or NULL: no rotation */
    int32_t interleaved;    /* rotated pairs: 0 = (i, i + d/2), 1 = (2i, 2i + 1) */
    const float *q_weight;  /* device [d], or NULL: queries are not normalised */
    const float *k_weight;  /* device [d], or NULL: keys are not normalised */
    float eps;              /* > 0 where a weight is given */
} ssa_kv_append_args;

/*
 * sparse_kv_append -- fills the cache that sparse_attn_decode (bf16) and sparse_attn_tree
 * read from a layer's projections, in one pass.  With P the token's position, per head:
 *   y = x * w / sqrt(mean(x^2) + eps)      (queries and keys whose weight is given)
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin), angle P * freqs[i], for pair i
 * values are stored as they come.  Everything is fp32, the angles fp64 until they are
 * reduced to one turn; one rounding at the end, to bf16 or to the cache's codes.
 * Errors: a null or misaligned pointer or a size out of range is SSA_ERR_INVALID, a head
 * dimension other than 64 or 128 or an unknown format SSA_ERR_UNSUPPORTED.  On the device,
 * SSA_ERR_INVALID goes to dev_status for a tok_ptr that descends or passes n_tokens, a
 * row outside the cache or a negative position; tokens without a valid row and position
 * are then skipped, the others written.  Nothing is looked at when n_tokens is 0.
 */
SSA_API int sparse_kv_append(const ssa_kv_cache *cache, const ssa_kv_append_args *args, int32_t *dev_status,
                             void *stream);

/*
 * sparse_kv_read -- reads cache rows back as bf16 (exactly the values they stand for): row
 * row0[b] + i of sequence b goes to token tok_ptr[b] + i of k_out and v_out, i <
 * tok_ptr[b+1] - tok_ptr[b].  The descriptors, padding and errors are those of
 * sparse_kv_append.  With head-major outputs of one sequence this gives the K and V that
 * sparse_attn_fwd takes.
 */
SSA_API int sparse_kv_read(const ssa_kv_cache *cache, int n_tokens, const int32_t *tok_ptr, const int32_t *row0,
                           const ssa_rows *k_out, const ssa_rows *v_out, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------ */
/* Attention of drafted trees over the cache                                        */
/* ------------------------------------------------------------------------------ */

#define SSA_TREE_MAX 64 /* nodes of a tree */

/*
 * The keys a tree can reach, per KV head: for heads h of the group, offsets
 * {r - t : r in D_h, 0 <= t < depth} (1 <= offset < S) and columns, merged over the
 * group's heads, with the lists as bitmaps beside them.  Made once per plan by
 * sparse_tree_lists; every pointer is a device buffer owned by the caller, sized from
 * ssa_tree_sizes:
 *   diag_bits, col_bits [n_heads][words] (uint64; bit x of the row = x is in the list),
 *   group_offs, group_cols [H_kv][words] (the merged lists as bitmaps),
 *   off_rank, col_rank [H_kv][words] (merged entries below 64 * word),
 *   off_ptr, col_ptr, head_ptr [H_kv + 1], heads [n_heads] (of each KV head, ascending),
 *   offs [max(n_off,1)][2], cols [max(n_col,1)][2]: the entry, and for the first 16 heads k of
 *   the group: offs bit k = all of offset .. offset + depth - 1 are diagonals of the head,
 *   bit 16 + k = some are; cols bits k and 16 + k = a column of the head
 */
typedef struct ssa_tree_sizes {
    int32_t n_heads;
    int32_t H_kv;
    int32_t S;
    int32_t depth;
    int32_t words;       /* 64-bit words per bitmap row: S / 64 + 2 */
    int32_t max_group;   /* most heads that share a KV head */
    int32_t max_entries; /* most offsets + columns of a KV head */
    int32_t reserved;
    int64_t n_off;
    int64_t n_col;
} ssa_tree_sizes;

typedef struct ssa_tree_lists {
    ssa_tree_sizes sizes;
    uint64_t *diag_bits;
    uint64_t *col_bits;
    uint64_t *group_offs;
    uint64_t *group_cols;
    int32_t *off_rank;
    int32_t *col_rank;
    int32_t *off_ptr;
    int32_t *offs;
    int32_t *col_ptr;
    int32_t *cols;
    int32_t *head_ptr;
    int32_t *heads;
} ssa_tree_lists;

/* Workspace bytes of either pass of sparse_tree_lists. */
SSA_API size_t sparse_tree_lists_ws_bytes(int n_heads, int H_kv, int S);

/*
 * sparse_tree_lists -- two passes, like sparse_pattern_extend.
 *   plan    from sparse_pattern_extend (its extended lists are read; a Case-2 plan is
 *           SSA_ERR_UNSUPPORTED)
 *   H_kv    KV heads; n_heads % H_kv == 0 when kv_map is NULL
 *   depth   [1, SSA_TREE_MAX]: the most nodes on one path of the trees to come (1 for
 *           single tokens)
 *   kv_map  device int32 [n_heads] or NULL (h / (n_heads / H_kv))
 *   sizes   host, filled when lists == NULL (sizing pass, which SYNCHRONISES `stream`)
 *   lists   non-NULL: fill pass, no synchronisation; lists->sizes must be those of the
 *           sizing pass.  Lists that no longer fit set SSA_ERR_CAPACITY in dev_status and
 *           are left empty (head_ptr, off_ptr and col_ptr 0): an attention with them writes
 *           nothing.
 * A kv_map entry outside [0, H_kv) is SSA_ERR_INVALID (sizing pass: returned).
 */
SSA_API int sparse_tree_lists(const ssa_plan *plan, int H_kv, int depth, const int32_t *kv_map,
                              ssa_tree_sizes *sizes, const ssa_tree_lists *lists, void *ws, size_t ws_bytes,
                              int32_t *dev_status, void *stream);

/*
 * sparse_attn_tree -- one step of drafted trees over a cache in any format, under the
 * extended mask.  Sequence b has len[b] committed rows and the nodes n < n_nodes[b], whose
 * keys and values lie in the rows len[b] + n (sparse_kv_append with row0 = len).  Node n
 * follows parent[b][n] (< n), or the committed tokens when that is -1; t_n is its depth
 * (0 in that case) and p_n = len[b] + t_n its position.  Its keys are
 *   {j < len : p_n - j in D_h or j in C_h}
 *   U {a = n or an ancestor of n : t_n - t_a in D_h or p_a in C_h}
 *   O[b][n][h] = sum softmax_j(scale * q . k_j) v_j,  LSE natural log
 * so that a node's result is the row that sparse_attn_decode gives once its path is
 * committed; one node per sequence is the ordinary decoding step, over a cache of any
 * format.  (Over a bf16 cache sparse_attn_decode does that step too.  It works head by head, this
 * call reads a key once for all heads of its group: take this one where they share keys, as
 * windows do -- 16 sequences, d = 64: 14 us against 25, 64 sequences 27 against 94 -- and
 * sparse_attn_decode for a few sequences whose heads have bands of their own -- d = 128, 1
 * sequence 13 us against 19 here, 4 sequences 25 against 26, 16 sequences 61 for both.)  No key:
 * O = 0, LSE = -inf.  A logit of -inf has no weight.  fp32 logits and statistics; weights of 11
 * bits at least, or to 2^-32 of a row's largest; bf16 O.  Values in rows that a query does not
 * retain do not touch it, NaN and infinities included.
 *
 *   Q, O      device bf16 [B][T][H_q][d], contiguous, 16-byte aligned (not the same buffer)
 *   T         [1, SSA_TREE_MAX];  B = cache->B
 *   len       device int32 [B];  n_nodes device int32 [B] or NULL (T each)
 *   parent    device int32 [B][T] or NULL (a chain: parent n - 1)
 *   lists     sizes.n_heads == H_q, sizes.H_kv and sizes.S as the cache's
 *   LSE       device float32 [B][T][H_q]
 * Rows of O and LSE of nodes n >= n_nodes[b] are left as they were.  A sequence with len < 0, a
 * node count outside [0, T], len + n_nodes > S, a parent not in [-1, n) or a path longer
 * than sizes.depth sets SSA_ERR_INVALID in dev_status and gets O = 0, LSE = -inf for its
 * nodes.  No workspace: the parts of a long key list are joined inside a thread-block
 * cluster, in a fixed order.  With more than 32 rows (heads of a group x T) a KV head the
 * kernel's waits are bounded: an expired one sets SSA_ERR_TIMEOUT in dev_status and leaves O and
 * LSE unspecified.
 */
SSA_API int sparse_attn_tree(const void *Q, const ssa_kv_cache *cache, int H_q, int T, const int32_t *len,
                             const int32_t *n_nodes, const int32_t *parent, const ssa_tree_lists *lists, float scale,
                             void *O, float *LSE, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------ */
/* Diagnostics                                                                     */
/* ------------------------------------------------------------------------------ */

/* Message of the last failing call on this thread ("" if none). */
SSA_API const char *ssa_last_error(void);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
SSA_API int ssa_version(void);

/*
 * Time limit, in nanoseconds, of every bounded wait inside the kernels that wait on
 * copies or tensor-core work (attention, averaged maps, capture, tree attention of more
 * than 32 rows a KV head; default 2e9; 0 makes a wait give up at its first unsuccessful
 * poll).  When a wait expires the kernel writes SSA_ERR_TIMEOUT to dev_status, drains its
 * own copies and tensor-core work in flight, frees its tensor memory and returns.
 * Process-wide; meant for fault-handling tests.
 * Returns the previous value.
 */
SSA_API int64_t ssa_set_wait_limit_ns(int64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* SSA_H */
