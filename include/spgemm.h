/*
 * spgemm.h -- C ABI of libspgemm.so: sparse general matrix-matrix product
 * C = A * B on CSR matrices, for one AMD Instinct MI355X (gfx950) GPU.
 *
 * Method (gMAGNUS page, "gMAGNUS: Fast SpGEMM on GPUs for Irregular Matrices
 * via Hierarchical Multisplit", §III, Algorithm 3):
 *   - rows whose intermediate product fits an on-chip accumulator ("light"
 *     rows, §II-B, §III-A) are computed row by row (Gustavson, Eq. 1) with LDS
 *     hash accumulators, binned by size (§III-E);
 *   - "heavy" rows are expanded by an outer product into an intermediate
 *     matrix C-hat (§III-B, Eq. 2), split by a hierarchical multisplit into
 *     column-range chunks (§III-C), and every chunk is accumulated entirely in
 *     LDS (dense accumulator for heavy chunks, hash for light ones, §III-E);
 *   - chunk count and levels come from C's column count and the LDS size
 *     (§III-D, Eq. 4-7).
 * The two-phase interface (symbolic computes C.rowPtr and nnz(C), numeric
 * fills C.col and C.val) follows §II-B of the same page and the
 * symbolic/numeric split described in §2 of the Ocean page.
 *
 * Conventions shared by every entry point
 *   - All matrix arrays are DEVICE pointers on the current HIP device; every
 *     size and count is a host integer.  `stream` is a hipStream_t passed as
 *     void* (NULL = the legacy default stream).
 *   - CSR: row_ptr (rows+1 entries, int32), col (nnz, int32), val (nnz, float
 *     or double per `dtype`).  Inputs must be canonical: row_ptr[0] == 0,
 *     row_ptr non-decreasing, 0 <= col < ncols, columns strictly increasing
 *     within a row.  opts->validate checks this on the device.
 *   - Output C is canonical CSR; an entry exists iff at least one stored
 *     pair A[i,k], B[k,j] exists (a computed 0.0 is kept).
 *   - Nothing is thrown across the ABI; every call returns spgemm_status.
 *   - Calls on one plan are not thread-safe; distinct plans are independent.
 */
#ifndef SPGEMM_H
#define SPGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum spgemm_status {
  SPGEMM_OK = 0,
  SPGEMM_ERR_INVALID_ARG = -1,    /* null pointer, negative size, bad dtype  */
  SPGEMM_ERR_INVALID_CSR = -2,    /* opts->validate found a non-canonical input */
  SPGEMM_ERR_INDEX_OVERFLOW = -3, /* int32 C.row_ptr requested, nnz(C) > INT32_MAX,
                                     or a size exceeds the int32 index range */
  SPGEMM_ERR_OOM = -4,            /* device allocation failed; C untouched   */
  SPGEMM_ERR_HIP = -5,            /* HIP runtime error; see spgemm_last_error */
  SPGEMM_ERR_STATE = -6,          /* call order violated or plan in error state */
  SPGEMM_ERR_INTERNAL = -7        /* a device-side capacity check tripped    */
} spgemm_status;

typedef enum spgemm_dtype {
  SPGEMM_F32 = 0, /* CSR values, logits, gradients */
  SPGEMM_F64 = 1, /* CSR values                    */
  SPGEMM_BF16 = 2, /* the expert layer's tensors   */
  SPGEMM_F16 = 3,
  SPGEMM_E4M3 = 4 /* weights of spgemm_expert_step   */
} spgemm_dtype;

/* Optional device allocator: return a device pointer of at least `bytes`
 * usable in stream order on `stream`, or NULL on failure.  With alloc == NULL
 * the library uses hipMallocAsync / hipFreeAsync on the plan's stream. */
typedef void *(*spgemm_alloc_fn)(size_t bytes, void *stream, void *ctx);
typedef void (*spgemm_free_fn)(void *ptr, void *stream, void *ctx);

/* Tuning and override knobs.  Zero-initialise, then set what you need; a zero
 * field means "automatic". */
typedef struct spgemm_options {
  int64_t lds_budget;           /* s_LM in bytes (gMAGNUS §III-D); 0 = LDS per
                                   work group of the device (160 KiB on gfx950) */
  int64_t heavy_threshold;      /* tau; 0 = derived from s_LM (Eq. 4 reading)   */
  int64_t dense_width;          /* final chunk width W (power of two); 0 = derived */
  int64_t mem_budget;           /* bytes for the heavy intermediate (the outer
                                   product and multisplit buffers, 8 (fp32) or
                                   12 (fp64) bytes per element, two buffers when
                                   there are levels); heavy rows are processed
                                   in batches of consecutive rows that fit it
                                   (at least one row a batch).  One batch keeps
                                   its expansion from symbolic to numeric;
                                   several batches expand again in numeric.
                                   0 = 45% of the device memory free at
                                   spgemm_symbolic, at least 1 GiB            */
  int32_t max_chunks_per_level; /* n_chunksMax (power of two >= 2); 0 = 32       */
  int32_t rowptr64;             /* 1: C.row_ptr is int64, else int32            */
  int32_t validate;             /* 1: check A and B are canonical CSR           */
  int32_t single_stream;        /* 1: light and heavy work on the caller's stream */
  int32_t profile;              /* 1: time each kernel phase with HIP events
                                   recorded on the stream it runs on; read the
                                   result from spgemm_stats.phase_ms           */
  int32_t histogram_from_data;  /* 1: count each level's (row, chunk) elements
                                   by reading the expanded columns (K6 as the
                                   gMAGNUS page prints it); 0: derive the same
                                   counts from the structure of A and of B's
                                   rows (default; the read pass is also used
                                   when n_req exceeds 8192)                    */
  spgemm_alloc_fn alloc;        /* optional allocator (see above)               */
  spgemm_free_fn free;
  void *alloc_ctx;
  int32_t expansion;            /* how the heavy rows' products reach their
                                   final chunks (the chunk tree, C and the
                                   parameters are the same in every mode):
                                   0 (default): one pass; every product
                                     is made from A and B row by row and
                                     written straight to its final chunk
                                     (needs the chunk counts from the
                                     structure and n_req <= 4096, else
                                     mode 2);
                                   1: as the gMAGNUS page prints it: masked
                                     CSC, outer product into C-hat, then one
                                     multisplit pass per level;
                                   2: the first multisplit level made from A
                                     and B row by row (C-hat never written),
                                     later levels as in mode 1              */
  int32_t heavy_row_threshold;  /* rows with more intermediate products than
                                   this take the heavy path; 0 = the
                                   heavy_threshold option if set, else
                                   floor(tau / 3): the largest light row whose
                                   numeric LDS table (2 slots per product)
                                   leaves room for three work groups per CU.
                                   Chunks keep tau (recursion, bins).        */
  int32_t light_hash_only;      /* 1: every light row takes the LDS hash
                                   accumulator; 0 (default): a light row whose
                                   products span at most 128 x its bin's
                                   product bound columns (at most 65536) takes
                                   the dense window: an LDS bitmap over the
                                   span, ranks by prefix popcount, values
                                   added at their rank (no hash, no sort);
                                   other rows of at least 512 products take a
                                   dense window over the 2048 columns around
                                   their diagonal position (row * n / m) plus
                                   an LDS hash table for the columns outside
                                   it, when those outliers fit half of the
                                   table (only the outliers are sorted)     */
  int32_t workflow;             /* how light rows get their output size (Ocean
                                   page, §3 and Table 1; heavy rows always take
                                   the exact chunk path):
                                   0 (default): symbolic pass (exact counts);
                                   1: upper bound: each light row reserves its
                                     product count P_i of output slots, is
                                     computed into them during
                                     spgemm_symbolic, and copied into C by
                                     spgemm_numeric;
                                   2: HyperLogLog estimate: per-B-row sketches
                                     merged per A row, min(P_i, ceil(coef*E))
                                     slots; rows that do not fit are computed
                                     again with P_i slots;
                                   3: choose by Table 1 (1 below 64 products
                                     per row, 2 when products / nnz(A) >= 8
                                     and the compression ratio of a 3% row
                                     sample is >= 8, else 0).
                                   C is the same in every mode. */
  int32_t hll_registers;        /* registers per sketch, 32 or 64; 0 = 32 when
                                   products / nnz(A) < 48, else 64          */
  int32_t hll_coef_pct;         /* estimate multiplier in percent; 0 = 200 with
                                   32 registers, 150 with 64               */
  int32_t light_no_esc;         /* 1: rows of at most 32 products take the LDS
                                   hash kernels; 0 (default): they take the
                                   expand-sort-compact kernel (32 lanes per
                                   row, sort by lane exchanges, no LDS;
                                   Ocean page, §3)                         */
  int64_t index_limit;          /* largest value accepted where an index is
                                   held in 32 bits: nnz(C) with an int32
                                   C.row_ptr, and a row's intermediate product
                                   count (its row-local product offsets are
                                   int32).  0 = INT32_MAX; a smaller value
                                   only serves tests of the overflow checks  */
  int64_t debug_device_error;   /* test hook, 0 in normal use: when nonzero,
                                   spgemm_numeric ends by storing this value
                                   in the plan's device status word on its
                                   stream, as a tripped device-side capacity
                                   check does, so that the reporting path
                                   (spgemm_wait, spgemm_get_stats) can be
                                   exercised from the host               */
  int64_t dense_direct;         /* 1: with expansion 0, dense chunks (W-wide
                                   slots of a heavy row holding more than
                                   min(tau, W/2) products) are accumulated
                                   straight from A and B (each entry's run of
                                   its B row inside the slot, found among B's
                                   per-slot runs) instead of from the expanded
                                   intermediate, which then holds only the
                                   light chunks' products; 0 (default): every
                                   product is expanded.  Same C either way.  */
  int64_t reserved[1];
} spgemm_options;

/* Parameters chosen by GetMagnusParams (gMAGNUS §III-D, Eq. 4-7). */
typedef struct spgemm_params {
  int64_t tau;              /* heavy threshold: a row/chunk is heavy iff its
                               element count exceeds tau                      */
  int64_t n_dense;          /* max dense accumulator width for numeric        */
  int64_t dense_width;      /* W = floor_pow2(n_dense): final chunk width     */
  int64_t chunks_required;  /* next_pow2(ceil(ncols / W)), at least 1         */
  int32_t chunks_max;       /* n_chunksMax                                    */
  int32_t levels;           /* multisplit levels (0 when chunks_required == 1) */
  int32_t v_chunks[8];      /* chunks per row at each level                   */
  int64_t level_width[8];   /* column width of a chunk after each level       */
} spgemm_params;

/* Kernel phases timed when spgemm_options.profile is set. */
typedef enum spgemm_phase {
  SPGEMM_PH_ROW_INFO = 0,        /* products per row, light/heavy bins (plan)   */
  SPGEMM_PH_SYM_LIGHT = 1,       /* light-row LDS hash symbolic                 */
  SPGEMM_PH_CSC = 2,             /* masked CSR->CSC and segment reservations   */
  SPGEMM_PH_OUTER_PRODUCT = 3,   /* C-hat expansion                             */
  SPGEMM_PH_HISTOGRAM = 4,       /* per-level (row, chunk) counts               */
  SPGEMM_PH_MULTISPLIT = 5,      /* per-level reorder into chunks              */
  SPGEMM_PH_SYM_CHUNK_HASH = 6,  /* light-chunk hash symbolic                   */
  SPGEMM_PH_SYM_CHUNK_DENSE = 7, /* heavy-chunk bitmap symbolic                 */
  SPGEMM_PH_ROWPTR = 8,          /* C.row_ptr scan and numeric binning          */
  SPGEMM_PH_NUM_LIGHT = 9,       /* light-row LDS hash numeric + sort           */
  SPGEMM_PH_NUM_CHUNK_HASH = 10, /* light-chunk hash numeric + sort             */
  SPGEMM_PH_NUM_CHUNK_DENSE = 11,/* heavy-chunk dense LDS numeric               */
  SPGEMM_PH_CHUNK_HIST = 12,     /* per-row W-wide chunk counts from structure  */
  SPGEMM_PH_EXPAND_SPLIT = 13,   /* first multisplit level fed from A and B     */
  SPGEMM_PH_EXPAND_FINAL = 14,   /* products made with values and written to
                                    their final chunks                          */
  SPGEMM_PH_SYM_HEAVY = 15,      /* heavy-row symbolic of the batched schedule,
                                    where values are not expanded in symbolic   */
  SPGEMM_PH_COUNT = 16
} spgemm_phase;

typedef struct spgemm_stats {
  int64_t products;           /* P = sum_i sum_{k in A_i} nnz(B_k); flops = 2P */
  int64_t max_row_products;
  int64_t light_rows;         /* rows with 0 < P_i <= tau                      */
  int64_t heavy_rows;         /* rows with P_i > tau                           */
  int64_t heavy_products;     /* P_h = nnz(C-hat)                              */
  int64_t heavy_a_nnz;        /* nnz of A restricted to heavy rows             */
  int64_t nnz_c;
  spgemm_params params;
  int64_t level_elems[8];     /* elements entering each multisplit level       */
  int64_t final_chunks;       /* non-empty chunks accumulated                  */
  int64_t dense_chunks;       /* of which in a dense LDS accumulator           */
  int64_t lds_hash_products;  /* products summed in LDS hash tables            */
  int64_t lds_dense_products; /* products summed in LDS dense accumulators     */
  int64_t global_products;    /* products summed in global memory (always 0)   */
  int64_t batches;            /* heavy-row batches (0 with no heavy rows)      */
  double ms_plan, ms_symbolic, ms_numeric; /* host wall time of each call      */
  double phase_ms[16];        /* GPU time of each spgemm_phase (with profile)  */
  int32_t phase_windows[16];  /* event-bracketed windows summed in phase_ms;
                                 a window holds one launch for the outer
                                 product, histogram, multisplit and dense
                                 phases (one per level for the per-level ones,
                                 and one per batch and expansion)           */
  int64_t device_errors;      /* device status bits seen (0 when all is well)  */
  int64_t heavy_row_threshold; /* rows above this many products were heavy     */
  int64_t chunk_col_bytes;    /* bytes of a column in the heavy intermediate:
                                 2 when it holds chunk-local 16-bit columns */
  int32_t workflow;           /* size prediction used (options.workflow 0-2) */
  int32_t hll_registers;      /* registers per sketch (workflow 2), else 0     */
  int64_t light_capacity;     /* output slots reserved for light rows (1, 2)   */
  int64_t overflow_rows;      /* light rows computed again with P_i slots      */
  double sampled_cr;          /* compression ratio of the row sample (mode 3)  */
  double phase_min_ms[16];    /* shortest window of each phase (with profile;
                                 0 for a phase with no window)              */
  int64_t hybrid_rows;        /* light rows accumulated in a dense window
                                 around their diagonal position plus an
                                 LDS hash table for the other columns     */
} spgemm_stats;

typedef struct spgemm_plan_s *spgemm_plan_t;
typedef struct spgemm_prune_s *spgemm_prune_t;

/* GetMagnusParams on the host; needs no GPU.  (gMAGNUS §III-D, Eq. 4-7.)
 * ncols = number of columns of C; lds_bytes = s_LM; val_bytes / col_bytes =
 * s_C.val / s_C.col; max_chunks_per_level = n_chunksMax (0 = 32);
 * dense_width = W override (0 = derived).  Where the printed formulas are
 * ambiguous, the readings taken are stated beside the code (params.cpp).
 * Errors: INVALID_ARG for non-positive sizes or a non-power-of-two
 * max_chunks_per_level / dense_width. */
spgemm_status spgemm_compute_params(int64_t ncols, int64_t lds_bytes,
                                    int32_t val_bytes, int32_t col_bytes,
                                    int32_t max_chunks_per_level,
                                    int64_t dense_width, spgemm_params *out);

/* Plan C = A * B (A: m x k, B: k x n).  Validates arguments, queries the
 * device, computes the parameters, counts intermediate products per row,
 * splits rows into light and heavy and bins them (gMAGNUS Algorithm 3,
 * setup phase).  Blocks once to read back the heavy count.  A and B are
 * borrowed until spgemm_destroy and must not change meanwhile.
 * Errors: INVALID_ARG, INDEX_OVERFLOW (nnz > INT32_MAX in an input),
 * INVALID_CSR (with validate), OOM, HIP; INDEX_OVERFLOW also when a row's
 * intermediate product count exceeds opts->index_limit (INT32_MAX).  On
 * error *out is NULL and nothing the caller owns was written. */
spgemm_status spgemm_plan(spgemm_plan_t *out, int64_t m, int64_t k, int64_t n,
                          const int32_t *dA_row_ptr, const int32_t *dA_col,
                          const void *dA_val, int64_t nnzA,
                          const int32_t *dB_row_ptr, const int32_t *dB_col,
                          const void *dB_val, int64_t nnzB, spgemm_dtype dtype,
                          const spgemm_options *opts, void *stream);

/* Symbolic phase: writes C.row_ptr (m+1 entries, int32, or int64 with
 * opts->rowptr64) into the caller's device buffer and returns nnz(C) on the
 * host (blocks once).  Heavy rows are expanded, multisplit and counted here;
 * the reordered intermediate is kept for numeric.  dC_row_ptr is written
 * last, only when the call succeeds.
 * Errors: STATE (not planned, or already run), INDEX_OVERFLOW (nnz(C) above
 * opts->index_limit, INT32_MAX by default, with an int32 C.row_ptr), OOM,
 * HIP, INVALID_CSR (with validate), INTERNAL (a device capacity check). */
spgemm_status spgemm_symbolic(spgemm_plan_t p, void *dC_row_ptr,
                              int64_t *nnzC);

/* Numeric phase: fills C.col (nnz(C) int32) and C.val (nnz(C), dtype),
 * columns sorted within each row.  Asynchronous on the plan's stream: the
 * kernels' own capacity checks (a numeric row or chunk whose size differs
 * from the symbolic count, a full hash table) are reported by spgemm_wait
 * or spgemm_get_stats, never by this call.  With a single heavy-row batch
 * (the symbolic expansion kept for numeric) this call allocates nothing, so
 * it cannot fail with OOM; with several batches each batch allocates its
 * chunk lists, and an OOM then leaves C.col/C.val partly written (C.row_ptr
 * from symbolic stays valid).
 * Errors: STATE (symbolic not run, or run twice), INVALID_ARG, OOM, HIP. */
spgemm_status spgemm_numeric(spgemm_plan_t p, int32_t *dC_col, void *dC_val);

/* Blocks until all work the plan has enqueued is done, then reports the
 * device status word: INTERNAL (with the check that tripped in
 * spgemm_last_error) when a device-side capacity check failed during
 * symbolic or numeric, in which case C must not be used; OK otherwise.  The
 * plan enters the error state on failure.  Call it (or spgemm_get_stats)
 * after spgemm_numeric before trusting C.
 * Errors: INVALID_ARG (NULL plan), INTERNAL, INVALID_CSR, HIP. */
spgemm_status spgemm_wait(spgemm_plan_t p);

spgemm_status spgemm_get_stats(spgemm_plan_t p, spgemm_stats *out);

/* Size prediction of the light rows (Ocean page, §3): after spgemm_symbolic
 * with options.workflow 1 or 2 (or 3 when it chose one of them), copies the
 * output slots reserved for every light row into dCap (m int64, device; 0
 * for other rows) and, with workflow 2, the HyperLogLog estimate of every
 * light row into dEst (m double, device).  Either pointer may be NULL.
 * Asynchronous on the plan's stream.  Errors: INVALID_ARG (NULL plan, dEst
 * without workflow 2), STATE (no symbolic yet, or workflow 0), HIP. */
spgemm_status spgemm_row_estimates(spgemm_plan_t p, int64_t *dCap, double *dEst);

/* Frees the plan's workspace (stream-ordered on the plan's stream). */
void spgemm_destroy(spgemm_plan_t p);

const char *spgemm_status_string(spgemm_status s);
/* Last error message of a plan, or of the calling thread when p == NULL. */
const char *spgemm_last_error(spgemm_plan_t p);

/* One Markov-clustering prune + column renormalisation of C (Trident page,
 * "Communication-Avoiding SpGEMM via Trident Partitioning", §5.7): keep
 * entries with C[i,j] >= threshold (compared in the value type), then divide
 * each kept entry by the fp64 sum of its column's kept entries, rounding once
 * to the value type.
 * Count call: computes the kept-entry row pointers into dOut_row_ptr (m+1;
 * int64 if out_rowptr64 else int32), the column sums, and returns the kept
 * count on the host (blocks once).  Fill call: writes dOut_col / dOut_val.
 * C is read through dC_row_ptr (int64 if c_rowptr64 else int32).
 * Errors: INVALID_ARG, INDEX_OVERFLOW, OOM, HIP, STATE. */
spgemm_status spgemm_prune_colnorm_count(
    spgemm_prune_t *out, int64_t m, int64_t n, const void *dC_row_ptr,
    int32_t c_rowptr64, const int32_t *dC_col, const void *dC_val,
    spgemm_dtype dtype, double threshold, void *dOut_row_ptr,
    int32_t out_rowptr64, int64_t *nnzOut, void *stream);
spgemm_status spgemm_prune_colnorm_fill(spgemm_prune_t p, int32_t *dOut_col,
                                        void *dOut_val);

/* The rest of one Markov-clustering iteration after the expansion C = A*A
 * (Trident page, §5.7: normalise the columns, prune entries below a
 * threshold, square the remaining entries).  With s_j the fp64 sum of all
 * entries of column j, y = C[i,j] / s_j is formed in fp64 and rounded once
 * to the value type (y = 0 when s_j = 0); entries with y >= threshold
 * (compared in the value type) are kept, with value y * y computed in the
 * value type.  Same two-call pattern, arguments, ownership and errors as
 * spgemm_prune_colnorm_count / _fill; the handle is released with
 * spgemm_prune_destroy. */
spgemm_status spgemm_mcl_inflate_count(
    spgemm_prune_t *out, int64_t m, int64_t n, const void *dC_row_ptr,
    int32_t c_rowptr64, const int32_t *dC_col, const void *dC_val,
    spgemm_dtype dtype, double threshold, void *dOut_row_ptr,
    int32_t out_rowptr64, int64_t *nnzOut, void *stream);
spgemm_status spgemm_mcl_inflate_fill(spgemm_prune_t p, int32_t *dOut_col,
                                      void *dOut_val);
void spgemm_prune_destroy(spgemm_prune_t p);

/* Transpose T = A^T of an m x n CSR matrix A into an n x m CSR matrix T, for
 * the rectangular products A * A^T that the Ocean page ("Ocean: Fast
 * Estimation-Based Sparse General Matrix-Matrix Multiplication on GPU",
 * evaluation on rectangular matrices) measures, and for restriction-type
 * operands (Trident page, §5.4).  T[j, i] = A[i, j] for every stored entry;
 * rows of T list their column indices in rising order (A's entries stored
 * row by row with rising rows; duplicates, if any, keep their storage
 * order), values are copied unchanged.
 * Inputs: dA_row_ptr (m+1; int64 if a_rowptr64 else int32), dA_col (nnz),
 * dA_val (nnz, float or double per dtype; NULL for the pattern only, then
 * dT_val is ignored).  Outputs, allocated by the caller: dT_row_ptr (n+1;
 * int64 if t_rowptr64 else int32), dT_col (nnz, int32), dT_val (nnz).
 * Temporaries (about 16 + 2*sizeof(value) bytes per entry) are allocated
 * with hipMallocAsync on `stream` and freed in stream order.  The call
 * blocks once, to read the device's column check.
 * Errors: INVALID_ARG (null pointer, negative size, bad dtype),
 * INDEX_OVERFLOW (m or n above INT32_MAX, or nnz above INT32_MAX with an
 * int32 dT_row_ptr), INVALID_CSR (a column index outside [0, n); T is then
 * undefined), OOM, HIP.  A's row pointers are trusted (row_ptr[0] == 0,
 * non-decreasing, row_ptr[m] == nnz). */
spgemm_status spgemm_transpose(int64_t m, int64_t n, int64_t nnz,
                               const void *dA_row_ptr, int32_t a_rowptr64,
                               const int32_t *dA_col, const void *dA_val,
                               spgemm_dtype dtype, void *dT_row_ptr,
                               int32_t t_rowptr64, int32_t *dT_col,
                               void *dT_val, void *stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * transpose, arguments, outputs and errors as spgemm_transpose, with the
 * temporaries taken from a fixed 64 MiB device array inside the library
 * instead of hipMallocAsync (each GPU the library runs on holds its own
 * array until the process ends).  The call makes no device allocation.
 * The caller still allocates T.  About 16 + 2 * sizeof(value) bytes per
 * entry are needed (fewer for narrow column ranges); a call whose
 * temporaries exceed 64 MiB returns INVALID_ARG (message in
 * spgemm_last_error(NULL)) without touching T.  Calls on one GPU share the
 * array: calls in stream order are safe (every piece that must start at
 * zero is cleared by a kernel on `stream`), calls that overlap on one GPU
 * (other streams or host threads) race.  Blocks once, as spgemm_transpose
 * does. */
spgemm_status spgemm_transpose_noalloc(int64_t m, int64_t n, int64_t nnz,
                                       const void *dA_row_ptr, int32_t a_rowptr64,
                                       const int32_t *dA_col, const void *dA_val,
                                       spgemm_dtype dtype, void *dT_row_ptr,
                                       int32_t t_rowptr64, int32_t *dT_col,
                                       void *dT_val, void *stream);

/* ---- The sparse expert layer ----------------------------------------------
 * A router picks k experts for every token: a sparse routing matrix R
 * (tokens x experts) whose row t holds the picked experts, columns rising,
 * and their weights.  Rows have k slots; a slot that holds no entry has
 * column -1 and value 0 and comes last, so with every slot taken (col, val)
 * and row_ptr[t] = t * k are R in CSR.  The experts' layer is the product
 * y_t = sum over row t of R[t,e] f_e(x_t).
 *
 * These calls are asynchronous on `stream`, allocate nothing and can be
 * captured in a graph.  Workspaces belong to the caller and hold nothing
 * between calls, but for the `kept` block that a forward pass leaves for its
 * backward pass. */

typedef struct spgemm_route_options {
  int32_t sigmoid;        /* scores: 0 softmax, 1 sigmoid (1 / (1 + exp(-z)))  */
  int32_t groups;         /* expert groups of equal size, 0 = 1, at most 64    */
  int32_t top_groups;     /* groups that may be picked from, 0 = all           */
  int32_t no_renormalise; /* 0: the weights of a row sum to `scale`            */
  float scale;            /* factor on the weights, 0 = 1                      */
} spgemm_route_options;

/* Routing: row t of dCol / dVal (T x k) from row t of the logits (T rows of E,
 * row stride ld elements; fp32, bf16 or fp16).
 *   key = z + bias (softmax) or sigmoid(z) + bias (sigmoid), in fp32; bias
 *   (E, fp32) may be NULL and only enters the keys.  An expert is out where
 *   its logit or key is minus infinity or NaN, and in rows whose byte of
 *   dActive (T, may be NULL) is 0, whatever such a row holds.
 *   Groups: the top_groups groups with the largest scores, a score being the
 *   group's largest key (softmax) or the sum of its two largest (sigmoid).
 *   Picked: the k largest keys left; of equal ones the lowest expert, and of
 *   equal groups the lowest.
 *   Weights: exp(z) over the sum of exp(z) of the picked experts, or, with
 *   no_renormalise, of all that are not out; sigmoid(z), divided by the
 *   picked ones' sum + 1e-20 unless no_renormalise.  Times scale.
 * Errors: INVALID_ARG (E outside [1, 1024], k outside [1, 64] or above the
 * experts of the chosen groups, groups that do not divide E, ld < E, bad
 * dtype, null arrays), INDEX_OVERFLOW (T * k above INT32_MAX), HIP. */
spgemm_status spgemm_route(int64_t T, int64_t E, int32_t k, const void *dLogits,
                           int64_t ld, spgemm_dtype dtype, const float *dBias,
                           const uint8_t *dActive,
                           const spgemm_route_options *opts, int32_t *dCol,
                           float *dVal, void *stream);

/* The gradient of the logits (T x E, contiguous, in the logits' type; every
 * element is written) for the gradient of the values (T x k).  dCol is what
 * spgemm_route gave for the same arguments; the scores are computed again. */
spgemm_status spgemm_route_backward(int64_t T, int64_t E, int32_t k,
                                    const void *dLogits, int64_t ld,
                                    spgemm_dtype dtype, const float *dBias,
                                    const spgemm_route_options *opts,
                                    const int32_t *dCol, const float *dGradVal,
                                    void *dGradLogits, void *stream);

/* Dispatch, the transpose of R: dRowPtr (E + 1) and dEntry (T * k), the
 * entries t * k + i of every expert in rising order.  Columns outside [0, E)
 * are no entries.  Work: spgemm_dispatch_workspace bytes. */
int64_t spgemm_dispatch_workspace(int64_t T, int32_t k, int64_t E);
spgemm_status spgemm_dispatch(int64_t T, int32_t k, int64_t E,
                              const int32_t *dCol, int32_t *dRowPtr,
                              int32_t *dEntry, void *dWork, int64_t work_bytes,
                              void *stream);

/* A kept_form that nothing but a caller who asks for it sets. */
#define SPGEMM_KEPT_E4M3 0x45344d33

/* An expert layer: x is T x D, w_in E x 2F x D (an expert's F gate rows, then
 * its F up rows), w_out E x D x F, all bf16 or fp16. */
typedef struct spgemm_experts_desc {
  int64_t tokens, experts, width, hidden; /* T, E, D, F                        */
  int64_t x_ld;        /* row stride of x in elements, at least D              */
  int64_t grad_ld;     /* row stride of grad_y (backward)                      */
  int32_t k;           /* slots of a row of R                                  */
  spgemm_dtype dtype;  /* SPGEMM_BF16 or SPGEMM_F16                            */
  int32_t unaligned;   /* 1: a base address is no multiple of 16 bytes         */
  int32_t kept_form;   /* SPGEMM_KEPT_E4M3: the kept block holds the rows of x
                          in 8 bits (spgemm_layer_norm_forward has the form),
                          about D bytes a token in place of 8 F an entry; any
                          other value: the pre-activations (this field was
                          reserved, and callers may have left it unset)        */
} spgemm_experts_desc;

/* Bytes of the kept block and of the two workspaces (any may be NULL).
 * Operands whose rows do not begin at 16-byte boundaries (D, F or a stride no
 * multiple of 8, or `unaligned`) are copied in every call, all experts' weights
 * too, and the copies counted.
 * Errors: INVALID_ARG (experts outside [1, 1024], k outside [1, 64], bad sizes,
 * strides or dtype), INDEX_OVERFLOW (sizes or strides beyond the kernels'
 * indexes or beyond one launch's 2^32 work items). */
spgemm_status spgemm_experts_sizes(const spgemm_experts_desc *desc,
                                   int64_t *kept, int64_t *forward_work,
                                   int64_t *backward_work);

/* y_t = sum over row t of w * W_out[e] (silu(W_gate[e] x_t) * (W_up[e] x_t)),
 * T x D contiguous; 0 for a row without entries.  Products and sums in fp32;
 * the hidden vector is rounded once to the tensors' type (in fp16 it has to
 * be below 65504), y once.  Columns outside [0, E) are no entries.  With dKept
 * (the sizes call's bytes) the pass leaves what the backward pass needs there. */
spgemm_status spgemm_experts_forward(const spgemm_experts_desc *desc,
                                     const void *dX, const void *dWIn,
                                     const void *dWOut, const int32_t *dCol,
                                     const float *dVal, void *dY, void *dKept,
                                     void *dWork, int64_t work_bytes,
                                     void *stream);

/* Gradients of x (T x D), w_in, w_out (in the tensors' type) and of the
 * values (T x k, fp32, 0 in empty slots), for the routing that the forward pass
 * was given (the kept block holds it).  With SPGEMM_KEPT_E4M3 they are the gradients at
 * the x that the 8 bits stand for, whose pre-activations are made again; dX is not
 * read then and may be NULL.  Every element is written: 0 for
 * experts without tokens.  Sums in fp32, in an order that only the routing
 * fixes: the same call gives the same bits.  The gradients of g and u, and
 * w * h, are rounded once to the tensors' type before their products; in fp16
 * in units of their row's or expert's largest magnitude, so that gradients and
 * values of any size keep the type's 11 bits.  The values' gradient is fp32
 * throughout. */
spgemm_status spgemm_experts_backward(
    const spgemm_experts_desc *desc, const void *dX, const void *dWIn,
    const void *dWOut, const void *dGradY, const void *dKept, void *dGradX,
    void *dGradWIn, void *dGradWOut, float *dGradVal, void *dWork,
    int64_t work_bytes, void *stream);

/* A whole expert layer for up to 16 tokens, as a decode step has them: logits,
 * routing and the experts' products in two launches. */
typedef struct spgemm_expert_step_desc {
  int64_t tokens, experts, width, hidden; /* T, E, D, F; T in [0, 16]; D and F
                                             at least 16                       */
  int64_t x_ld;              /* row stride of x in elements, at least D        */
  int32_t k;
  spgemm_dtype dtype;        /* of x and y: SPGEMM_BF16 or SPGEMM_F16          */
  spgemm_dtype weight_dtype; /* of w_in and w_out: dtype or SPGEMM_E4M3        */
  spgemm_dtype router_dtype; /* dtype or SPGEMM_F32                            */
  spgemm_route_options route;
} spgemm_expert_step_desc;

/* z = router x (router E x D; sums in 64 bits, rounded to fp32), then dCol and
 * dVal (T x k) as spgemm_route gives them for z, then y (T x D, contiguous) as
 * spgemm_experts_forward does; the columns are the routing's, so that y is the
 * layer's whole result.  All arrays but x are contiguous; any alignment that their
 * elements have, dWork at a multiple of 4 bytes.
 * With SPGEMM_E4M3 an expert's weight is W[r, c] = w[r, c] s[r / 128, c / 128]:
 * dInScale is E x ceil(2F / 128) x ceil(D / 128), dOutScale E x ceil(D / 128) x
 * ceil(F / 128), fp32; else they are not read.  The 8-bit values are multiplied as
 * they are, in x's type, and the scales applied in fp32 to the sums over 64
 * columns.  Products and sums in fp32, in an order that the sizes and the picked
 * experts fix; the hidden vector is held in two terms of x's type, 16 or 22 bits (fp16: to
 * 2^-36 below 2^-14; a value beyond the type is infinite: in fp16 it has to be
 * below 65520), y is rounded once.
 * Errors: INVALID_ARG (as spgemm_route; more than 16 tokens; a width below 16; types, strides, null
 * arrays, a workspace too small), INDEX_OVERFLOW (a width above 2^20), HIP. */
spgemm_status spgemm_expert_step_workspace(const spgemm_expert_step_desc *desc,
                                            int64_t *bytes);
spgemm_status spgemm_expert_step(
    const spgemm_expert_step_desc *desc, const void *dX, const void *dRouter,
    const float *dBias, const uint8_t *dActive, const void *dWIn,
    const float *dInScale, const void *dWOut, const float *dOutScale, void *dY,
    int32_t *dCol, float *dVal, void *dWork, int64_t work_bytes, void *stream);

/* The global norm of `count` tensors (fp32, bf16 or fp16, mixed at will) and
 * its clipping: norm = sqrt(sum g^2) in fp64, rounded into dNorm (1 fp32);
 * out = g * min(1, max_norm / (norm + 1e-6)) in fp64, rounded to fp32 and then
 * to out's type; right also where the norm itself is beyond fp32 (and infinite
 * in dNorm).
 * out[i] may be grads[i] itself; other overlaps are not allowed.  A norm that
 * is NaN makes every output NaN.  The tables of pointers, sizes (elements) and
 * types are host arrays, read during the call.
 * Errors: INVALID_ARG (null arrays, negative sizes, bad types, max_norm
 * negative or NaN, a workspace too small), INDEX_OVERFLOW, HIP. */
int64_t spgemm_clip_grad_norm_workspace(int64_t count);
spgemm_status spgemm_clip_grad_norm(int64_t count, const void *const *dGrads,
                                    void *const *dOut, const int64_t *sizes,
                                    const int32_t *grad_types,
                                    const int32_t *out_types, double max_norm,
                                    float *dNorm, void *dWork,
                                    int64_t work_bytes, void *stream);

/* ---- Layer norm, and rows kept in 8 bits ----------------------------------
 * As the calls of the expert layer: asynchronous on `stream`, no allocation,
 * workspaces and kept blocks of the caller. */

typedef struct spgemm_layer_norm_desc {
  int64_t rows, width;       /* T, D; D in [1, 16384]                          */
  int64_t x_ld, grad_ld;     /* row strides of x and grad_y in elements, >= D  */
  spgemm_dtype dtype;        /* of the rows: SPGEMM_F32, _BF16 or _F16         */
  spgemm_dtype weight_dtype; /* of weight and bias: SPGEMM_F32 or dtype        */
  float eps;                 /* >= 0                                           */
  int32_t kept_form;         /* 0 nothing, 1 statistics, 2 rows in 8 bits too  */
} spgemm_layer_norm_desc;

/* Bytes of the kept block and of the backward pass's workspace (either may be
 * NULL).  Errors of all three: INVALID_ARG (sizes, strides, types, eps,
 * kept_form, null arrays, a workspace too small), INDEX_OVERFLOW, HIP. */
spgemm_status spgemm_layer_norm_sizes(const spgemm_layer_norm_desc *desc,
                                      int64_t *kept, int64_t *backward_work);

/* y = (x - m) r w + b with m the row's mean and r = 1 / sqrt(v + eps), v the mean
 * of (x - m)^2; y is T x D, contiguous, in x's type, rounded once.  w and b have D
 * elements, b may be NULL.  Any alignment and stride.  kept_form 1 leaves m and r
 * (fp32) in dKept; 2 also the rows of x in 8 bits, by blocks of 128 columns: with
 * s the smallest power of two for which max |x| <= 448 s over the block's finite
 * values, no smaller than 2^-15 (fp16) or 2^-117, x / s rounded to e4m3 (nearest,
 * ties to even; at most 240 where s is 2^8, fp16, or 2^120); what is not finite
 * is held as NaN.  The sums of x and of (x - m)^2 have to be in fp32's range. */
spgemm_status spgemm_layer_norm_forward(const spgemm_layer_norm_desc *desc,
                                        const void *dX, const void *dWeight,
                                        const void *dBias, void *dY, void *dKept,
                                        void *stream);

/* With n = (x - m) r and a = dy w: dx = r (a - mean(a) - n mean(a n)) (T x D,
 * contiguous, in x's type), dw = sum over rows of dy n and db = sum over rows of
 * dy (dGradBias may be NULL) in the weights' type.  m and r are the kept ones; x
 * is the tensor (kept_form 1) or what its 8 bits stand for (2; dX is not read and
 * may be NULL; n is then off by up to 2^-4 |x| r, which for a mean of 16 deviations
 * is a whole one).  Sums in fp32, in an order that the sizes alone fix.  Without rows
 * dw and db are 0, and of the inputs only dWeight may not be NULL. */
spgemm_status spgemm_layer_norm_backward(
    const spgemm_layer_norm_desc *desc, const void *dX, const void *dWeight,
    const void *dGradY, const void *dKept, void *dGradX, void *dGradWeight,
    void *dGradBias, void *dWork, int64_t work_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SPGEMM_H */
