/*
 * Load-balanced CSR sparse matrix-vector product for one GB300 (sm_103a).
 *
 *     y = alpha * A * x + beta * y
 *
 * A is an m-by-n matrix in CSR form with int32 indices and fp32 or fp64
 * values.  CSR as defined on the Row-grouped CSR page ("New Row-grouped CSR
 * format for storing the sparse matrices on GPU with implementation in CUDA",
 * section 3, Figure 1): the nonzeros are stored row by row in `vals` with
 * their column indices in `col_idx`; `row_ptr` has m+1 entries, row i owns
 * positions row_ptr[i] .. row_ptr[i+1]-1, and row_ptr[m] = nnz.  The same
 * three arrays are the SpMV kernel's inputs in the load-balancing paper
 * (Osama, Porumbescu, Owens, "A GPU load-balancing programming model",
 * section 4.3, Listing 3), which computes each y entry as the row's sum of
 * values[nz] * x[indices[nz]].
 *
 * The library works in two steps.  spmv_plan_create analyses the row
 * lengths on the GPU (statistics by length class, after OpSparse's row
 * binning, section 5.1), chooses a kernel, and precomputes its schedule --
 * for the default merge-path kernel, the exact split of the m + nnz units
 * of work (every row end and every nonzero, "A GPU load-balancing
 * programming model", section 5.2.1) into equal tiles.  spmv_execute then
 * runs the product on a stream with no allocation and no synchronisation.
 *
 * All array arguments are DEVICE pointers (for example from torch CUDA
 * tensors) on the current CUDA device, except where a function says HOST.
 * Streams are cudaStream_t handles; NULL is the legacy default stream.
 * Every function returns an spmv_status_t; spmv_last_error() gives a
 * one-line description of the last failure on the calling thread.
 */
#ifndef LBCSR_SPMV_H
#define LBCSR_SPMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
/* a cudaStream_t */
typedef struct CUstream_st *spmv_stream_t;

typedef struct spmv_plan_s *spmv_plan_t;

typedef enum { SPMV_F32 = 0, SPMV_F64 = 1 } spmv_dtype_t;

typedef enum {
    SPMV_OK = 0,
    SPMV_ERR_INVALID_ARG = 1, /* null pointer, negative size, size limits, bad option */
    SPMV_ERR_INVALID_CSR = 2, /* row_ptr[0] != 0, row_ptr decreasing, row_ptr[m] != nnz,
                                 or a column index outside [0, n) */
    SPMV_ERR_ALLOC = 3,       /* device or host allocation failed in plan creation */
    SPMV_ERR_CUDA = 4,        /* a CUDA call or kernel launch failed */
    SPMV_ERR_UNSUPPORTED = 5  /* device is not sm_103 / option not available */
} spmv_status_t;

/* Kernels a plan can run. */
typedef enum {
    SPMV_KERNEL_AUTO = 0,       /* let the plan choose from the row-length statistics */
    SPMV_KERNEL_MERGE_PATH = 1, /* equal shares of rows + nonzeros per warp tile, fused carry-out fix-up */
    SPMV_KERNEL_THREAD_ROW = 2, /* one thread per row */
    SPMV_KERNEL_RGCSR = 3,      /* Row-grouped CSR (interleaved copy of A built by the plan);
                                   long rows, if any, by the long-row kernel */
    SPMV_KERNEL_LONG_ROWS = 4,  /* long rows by the long-row kernel (one warp per segment of
                                   4096 nonzeros), the other rows one thread per row */
    SPMV_KERNEL_RGCSR_SORTED = 5,/* Row-grouped CSR (groups of 32) over the rows listed, in
                                   each window of 1024 rows, by decreasing length, which
                                   cuts the padding; long rows by the long-row kernel */
    SPMV_KERNEL_GROUP_MAPPED = 6 /* group-level schedule ("A GPU load-balancing programming
                                   model", section 5.2.3): a CTA per 256 rows, their
                                   nonzeros shared by the CTA's threads */
} spmv_kernel_t;

/* Options for spmv_plan_create_ex; zero-initialise and set what you need. */
typedef struct {
    int32_t kernel;           /* spmv_kernel_t; SPMV_KERNEL_AUTO (0) = choose */
    int32_t items_per_thread; /* merge-path work items (rows + nonzeros) per
                                 thread; a tile is one warp, T = 32 * items.
                                 0 = chosen from the statistics (8-24).
                                 Allowed: 8, 12, 16, 24, 32 */
    int32_t rgcsr_group;      /* Row-grouped CSR group size G; 0 = chosen from
                                 the statistics (the largest G whose padding
                                 is at most 10 %, else the least padded).
                                 Allowed: 32, 64, 128, 256 */
    int32_t long_row_min;     /* Row-grouped CSR and long-row kernels: rows with
                                 at least this many nonzeros count as long and
                                 go to the long-row kernel; 0 = default (512).
                                 Allowed: 0 or >= 32 */
    int32_t with_spmm;        /* nonzero: also prepare spmv_execute_multi (the
                                 merge-path partition and its scratch, about
                                 1 KB per warp slot for fp32, 2 KB for fp64) */
    int32_t with_transpose;   /* nonzero: also prepare spmv_execute_transposed
                                 (the plan builds A^T in CSR form, 12-16 bytes
                                 per nonzero, and a plan for it) */
} spmv_options_t;

/*
 * Row-length statistics measured by the plan.  hist[k] counts rows whose
 * length falls in class k: class 0 = empty rows, class k >= 1 = lengths in
 * [2^(k-1), 2^k).  rg_slots[g] = storage (slots) a Row-grouped CSR layout
 * with group size 32 << g would need (each group padded to its longest
 * row).  bandwidth: the largest |column - row| over every row's first and
 * last stored nonzero.  flags: bit0 row_ptr[0] != 0, bit1 row_ptr
 * decreases, bit2 row_ptr[m] != nnz, bit3 a column index outside [0, n).
 */
typedef struct {
    int64_t hist[32];
    int64_t sum_len;
    int64_t rg_slots[4];
    int32_t min_len;
    int32_t max_len;
    int32_t n_empty;
    int32_t flags;
    int32_t bandwidth;
    int32_t reserved;
} spmv_row_stats_t;

typedef struct {
    int32_t m, n, nnz;
    int32_t dtype;                /* spmv_dtype_t */
    int32_t kernel;               /* spmv_kernel_t actually used */
    int32_t threads_per_tile;     /* merge-path kernel: one warp per tile */
    int32_t items_per_thread;     /* merge-path kernel */
    int32_t rgcsr_group;          /* Row-grouped CSR kernel */
    int64_t items_per_tile;       /* merge-path tile T = threads * items (rows + nonzeros) */
    int64_t num_tiles;            /* merge-path tiles P = ceil((m + nnz) / T), at least 1 */
    int32_t num_long_rows;        /* rows handled by the long-row kernels */
    int32_t launches_per_execute; /* kernel launches one spmv_execute issues */
    int64_t workspace_bytes;      /* device memory the plan owns */
    spmv_row_stats_t stats;
    int32_t long_row_min;         /* threshold of the long-row kernel (0 if unused) */
    int32_t long_segment_nnz;     /* nonzeros per long-row segment (one warp each) */
    int64_t num_long_segments;    /* segments over all long rows */
    int64_t rgcsr_slots;          /* slots of the Row-grouped copy (group_ptr[last]) */
    int32_t transposed_kernel;    /* spmv_kernel_t of the plan for A^T (-1: none) */
    int32_t transposed_launches;  /* kernel launches one spmv_execute_transposed issues */
    int64_t merge_path_warps;     /* merge-path kernel: warps W, each owning a contiguous run of
                                     about num_tiles / W tiles (for 16-byte aligned arrays; 0 when
                                     the plan runs another kernel) */
} spmv_plan_info_t;

/* What spmv_plan_export copies out. */
typedef enum {
    SPMV_EXPORT_PARTITION = 0,   /* int32 pairs (row, nonzero), num_tiles + 1 of them */
    SPMV_EXPORT_RG_GROUP_PTR = 1,/* int64[ceil(m/G) + 1] */
    SPMV_EXPORT_RG_ROW_LEN = 2,  /* int32[m] by position: row length, -1 for a row left to the
                                    long-row kernel */
    SPMV_EXPORT_RG_COL = 3,      /* int32[group_ptr[last]] */
    SPMV_EXPORT_RG_VAL = 4,      /* value type [group_ptr[last]] */
    SPMV_EXPORT_LONG_ROWS = 5,   /* int32[num_long_rows], ascending */
    SPMV_EXPORT_LONG_SEG_BEGIN = 6,/* int64[num_long_rows + 1]: first segment of each long row */
    SPMV_EXPORT_RG_PERM = 7,     /* int32[m]: the row at each position of the window-sorted copy */
    SPMV_EXPORT_T_PTR = 8,       /* int32[n + 1]: A^T in CSR form, row pointers */
    SPMV_EXPORT_T_IDX = 9,       /* int32[nnz]: its column indices (rows of A) */
    SPMV_EXPORT_T_VALS = 10,     /* value type [nnz] */
    SPMV_EXPORT_T_SRC = 11       /* int32[nnz]: each entry's position in A */
} spmv_export_t;

/*
 * Build a plan for A (device arrays row_ptr[m+1], col_idx[nnz], vals[nnz]).
 *
 * Limits: m >= 0, n >= 0, 0 <= nnz, m + nnz < 2^31.  When nnz > 0 the
 * pointers must be non-null; row_ptr must be non-null when m >= 0.
 * Ownership: the plan BORROWS row_ptr, col_idx and vals; they must stay
 * allocated and unchanged until spmv_plan_destroy (values may change if
 * spmv_plan_update_values is called afterwards).  The plan OWNS one device
 * workspace, allocated here and freed by spmv_plan_destroy.
 * Synchronisation: runs its analysis kernels on `stream` and waits for that
 * stream once (to read the ~0.4 KB statistics back) -- three times for the
 * Row-grouped CSR and long-row kernels, whose layouts are sized on the
 * device (long-row count, segment count, Row-grouped slots) before their
 * last allocation.  Results are synchronous.
 * Errors: INVALID_ARG for bad sizes/pointers; INVALID_CSR when the analysis
 * finds a malformed row_ptr or a column index outside [0, n); ALLOC; CUDA;
 * UNSUPPORTED when the current device is not compute capability 10.3.
 * On error *out is set to NULL and nothing is leaked.
 * Environment, read at each creation: SPMV_LOG=1 prints one line per plan
 * on stderr (the row statistics, the kernel and the rule that chose it);
 * SPMV_FORCE_KERNEL (a kernel name) and SPMV_ITEMS_PER_THREAD override the
 * choice when the options leave it open; SPMV_FAULT=alloc:N|launch:N makes
 * the N-th device allocation or launch step of the call fail, for testing
 * the clean-up paths.
 */
spmv_status_t spmv_plan_create(spmv_plan_t *out, int32_t m, int32_t n, int32_t nnz,
                               const int32_t *row_ptr, const int32_t *col_idx, const void *vals,
                               spmv_dtype_t dtype, spmv_stream_t stream);

/* As spmv_plan_create, with options (NULL = defaults). */
spmv_status_t spmv_plan_create_ex(spmv_plan_t *out, int32_t m, int32_t n, int32_t nnz,
                                  const int32_t *row_ptr, const int32_t *col_idx, const void *vals,
                                  spmv_dtype_t dtype, const spmv_options_t *options,
                                  spmv_stream_t stream);

/*
 * y = alpha * A * x + beta * y on `stream` (device x[n], y[m] of the plan's
 * value type).  alpha and beta are rounded to the value type.  If beta == 0
 * y is write-only: its old contents (NaN included) are not read.  x and y
 * must not overlap.  Asynchronous: returns after queueing the kernels; no
 * allocation, no host synchronisation.  A plan must not run on two streams
 * at once (its workspace holds per-execution carry state).
 * Errors: INVALID_ARG (null plan, or null x/y when the sizes need them),
 * CUDA (launch failure).
 */
spmv_status_t spmv_execute(spmv_plan_t plan, double alpha, const void *x, double beta, void *y,
                           spmv_stream_t stream);

/*
 * The same product with x and y in HOST memory (x_host[n], y_host[m] of
 * the plan's value type): on `stream`, copy x_host into the caller's
 * device buffer x_dev[n] (and y_host into y_dev[m] when beta != 0), run
 * spmv_execute(plan, alpha, x_dev, beta, y_dev, stream), and copy y_dev
 * back into y_host -- one cudaMemcpyAsync per copy.  Asynchronous like
 * spmv_execute: y_host holds the result once the stream has passed the
 * last copy (synchronise the stream before reading it).  For copies that
 * overlap other work the host buffers should be page-locked
 * (cudaHostAlloc, or pinned torch tensors); pageable memory also works.
 * x_dev and y_dev must not overlap each other or the plan's arrays.
 * Allocates nothing.  This is the call an application with its vectors on
 * the host makes; the product itself is the one above.
 * Errors: as spmv_execute, INVALID_ARG also for a null host or device
 * buffer the sizes need, CUDA when a copy cannot be queued.
 */
spmv_status_t spmv_execute_host(spmv_plan_t plan, double alpha, const void *x_host, double beta, void *y_host,
                                void *x_dev, void *y_dev, spmv_stream_t stream);

/*
 * Y = alpha * A * X + beta * Y for k right-hand sides ("A GPU
 * load-balancing programming model", section 4.3, Listing 4: the row loop
 * of SpMV with an inner loop over the columns of a dense matrix).  X is
 * n-by-k and Y m-by-k, device, row-major with leading dimensions ldx >= k
 * and ldy >= k (element (c, t) of X at X[c*ldx + t]); value type of the
 * plan.  alpha and beta as for spmv_execute (beta == 0: Y is write-only).
 * X and Y must not overlap.  The plan must have been created with
 * options.with_spmm != 0 (it then holds the merge-path partition, and the
 * long-row lists the paths below need).
 *
 * The call takes the first path that applies: (1) over the plan's
 * Row-grouped copy (groups of 32; long rows the copy leaves out, if at
 * most one per 4096 rows, by a warp per 4096-nonzero segment), in slices
 * of 32 (fp32) or 16 (fp64) columns; (2) for matrices whose rows have at
 * most 64 nonzeros, or with rows of 65 or more at most one per 4096 rows
 * and k <= 64 (fp32) / 32 (fp64): a warp per 32 rows straight from CSR,
 * long rows by a warp per segment -- both need k a multiple of 16 bytes'
 * worth of values and X, Y 16-byte aligned row by row; (3) otherwise the
 * merge-path partition, 128 columns per launch.  Every path gives the
 * same sums up to rounding order; none allocates; asynchronous.  A plan
 * must not run two products at once.
 * Errors: INVALID_ARG (null plan or pointers, k < 0, ld < k, plan without
 * with_spmm), CUDA (launch failure).  k == 0 or m == 0 is a no-op.
 */
spmv_status_t spmv_execute_multi(spmv_plan_t plan, int32_t k, double alpha, const void *X, int64_t ldx,
                                 double beta, void *Y, int64_t ldy, spmv_stream_t stream);

/*
 * y = alpha * A^T * x + beta * y: x has m entries, y has n (device, plan's
 * value type).  The plan must have been created with
 * options.with_transpose != 0: it then holds A^T in compressed-row form
 * (A in compressed-column form, the CSC of "A GPU load-balancing
 * programming model", section 4.1), each column's entries in increasing
 * row order, built by a stable radix sort on the GPU, and a plan of its own
 * for it (statistics, kernel choice, schedule), whose product this runs.
 * Semantics, synchronisation and errors as for spmv_execute.
 */
spmv_status_t spmv_execute_transposed(spmv_plan_t plan, double alpha, const void *x, double beta, void *y,
                                      spmv_stream_t stream);

/*
 * Point the plan at new values with the same sparsity pattern (vals[nnz],
 * device).  Plans that keep a reordered copy of the values (the
 * Row-grouped CSR kernel, A^T) repack it on `stream`; the others only
 * record the pointer.  Same ownership rule as at creation.
 */
spmv_status_t spmv_plan_update_values(spmv_plan_t plan, const void *vals, spmv_stream_t stream);

/* Free the plan's workspace (waits for the device to finish using it). NULL is a no-op. */
spmv_status_t spmv_plan_destroy(spmv_plan_t plan);

/* Fill *info (HOST) with the plan's sizes, chosen kernel and statistics. */
spmv_status_t spmv_plan_info(spmv_plan_t plan, spmv_plan_info_t *info);

/*
 * Copy one of the plan's internal arrays into HOST memory dst of `bytes`
 * bytes (for tests and inspection; synchronous).  INVALID_ARG if the plan
 * does not hold that array or bytes is smaller than its size; the size is
 * written to *needed when needed != NULL.
 */
spmv_status_t spmv_plan_export(spmv_plan_t plan, spmv_export_t what, void *dst, size_t bytes,
                               size_t *needed);

/*
 * One product y = alpha * A * x + beta * y that allocates nothing: no plan,
 * no cudaMalloc/cudaFree, no allocating library call.  The pages have no
 * counterpart; this entry point exists for callers that cannot allocate
 * device memory when they need a product -- for example a service that
 * hands the whole device to its own memory pool at start-up (a cudaMalloc
 * would fail or fragment the pool), or a latency-critical loop where a
 * cudaMalloc would synchronise the device and stall work queued on other
 * streams.
 *
 * Arguments as spmv_plan_create plus spmv_execute (device arrays, the
 * caller's stream).  It runs the merge-path kernel (tiles of 384 rows plus
 * nonzeros) with its scratch in one fixed-size array (about 6 MB) inside the
 * library's device image, which every GPU that loads the library holds
 * until the process exits.  Limit: m + nnz <= 2^28 = 268,435,456; larger
 * sizes return SPMV_ERR_INVALID_ARG.  The matrix is NOT checked (use
 * spmv_plan_create once to validate it); invalid indices give undefined
 * results.  All calls share the scratch array and each call clears what must
 * start at zero, so calls that overlap on the GPU (two streams, two host
 * threads) race.  Every call looks up the array's device address (a host
 * table lookup once the library's module is loaded on the device); the first
 * call on a device loads that module, so make it before any stream capture.
 * Asynchronous otherwise.  A tile copy that does not complete within about a
 * second stops that part of the product and sets a flag that
 * spmv_noalloc_device_status reports.  Returns SPMV_OK, SPMV_ERR_INVALID_ARG
 * or SPMV_ERR_CUDA (no message is set for spmv_last_error).
 */
spmv_status_t spmv_execute_noalloc(int32_t m, int32_t n, int32_t nnz, const int32_t *row_ptr,
                                   const int32_t *col_idx, const void *vals, spmv_dtype_t dtype,
                                   double alpha, const void *x, double beta, void *y,
                                   spmv_stream_t stream);

/*
 * Kernel-side failure flags of the last spmv_execute_noalloc on the current
 * device (HOST *flags; waits for the whole device, so not during a stream
 * capture; allocates nothing).  0 = no failure; bit 0: a tile copy did not
 * complete within about a second, and that product's y is incomplete.  The
 * pages have no counterpart.  Returns SPMV_OK, SPMV_ERR_INVALID_ARG or
 * SPMV_ERR_CUDA.
 */
spmv_status_t spmv_noalloc_device_status(int32_t *flags);

/*
 * Kernel-side failure flags of a plan (HOST *flags; waits for the device).
 * 0 = no failure.  Bit 0: a kernel's wait for its tile copies ran past its
 * time limit (about a second); the kernel then stopped that part of the work
 * instead of waiting forever, so the y of that product is incomplete.
 * Bit 2 (value 4), debug build only (libspmv_debug.so, compiled with
 * -DSPMV_DEBUG): an SpMV kernel met a column index outside [0, n) -- an
 * array changed after the plan was created, which the plan borrows
 * unmodified -- and gathered x[0] in its place; that y is wrong.  The
 * release build does not check (creation validates every index once).
 */
spmv_status_t spmv_plan_device_status(spmv_plan_t plan, int32_t *flags);

/*
 * Diagnostic: the ceiling of the x gather for a column pattern, by load
 * path.  The Row-grouped CSR page (sections 3 and 4) names the gather of x
 * as what limits SpMV once the matrix stream is coalesced (x through the
 * texture cache gave 1.3-1.8x); this call measures how fast each of the
 * GPU's load paths can gather x[col_idx[k]] for k = 0 .. nnz-1, with no
 * matrix values and no floating-point work, so that a kernel's time can be
 * set against the best one.
 *
 * path (spmv_gather_path_t): STREAM reads col_idx only; L1 gathers through
 * the read-only path (ld.global.nc); L2 through L2 only (ld.global.cg);
 * BULK16 by one 16-byte Tensor Memory Accelerator copy per gather into
 * shared memory; TMA4 by tile::gather4 tensor copies (x viewed as rows of
 * 32 bytes, four rows per instruction); L1_TMA4 half by L1, half by TMA4;
 * L1_TMA4_QUARTER three quarters by L1, one by TMA4; TMA4_16 as TMA4 over
 * rows of 16 bytes.  Three paths also stream the values vals[nnz] (device,
 * dtype) beside the L1 gathers, to measure what bringing in the matrix
 * costs the gathers: STREAM_LDG by coalesced loads, STREAM_BULK by one bulk
 * copy per 256 nonzeros and array into shared memory, STREAM_CPASYNC by
 * 16-byte cp.async (both need col_idx and vals 16-byte aligned),
 * STREAM_LDG_OCC as STREAM_LDG with the staged paths' shared memory reserved
 * (as many warps per SM), STREAM_LDG_STS by coalesced loads that the lanes
 * store to shared memory and read back, STREAM_LDG_FEW as STREAM_LDG with no
 * shared memory but only as many CTAs per SM as the staged paths fit,
 * STREAM_LDG_RES_1 .. _6 as STREAM_LDG with 4 CTAs per SM and 32, 64, ...,
 * 192 KB of shared memory reserved per SM (the L1 left to the gathers);
 * their checksum adds the values' bit patterns too.
 * col_idx[nnz] (device, int32, each in [0, n)), x[n] (device, dtype; 16-byte
 * aligned for the copy paths, BULK16 to TMA4_16, which also need
 * n * sizeof(value) >= 32).  *checksum (device uint64, zeroed by the caller) receives the sum,
 * modulo 2^64, of the bit patterns of the gathered values (the same for
 * every path except STREAM, which sums the columns instead).  *error
 * (device int32, zeroed by the caller): bit 0 is set if a copy did not
 * complete within about a second.  Asynchronous on `stream`; allocates
 * nothing.  Errors: INVALID_ARG; UNSUPPORTED when x is misaligned for the
 * path or the tensor-map encoder is unavailable; CUDA on launch failure.
 */
typedef enum {
    SPMV_GATHER_STREAM = 0,
    SPMV_GATHER_L1 = 1,
    SPMV_GATHER_L2 = 2,
    SPMV_GATHER_BULK16 = 3,
    SPMV_GATHER_TMA4 = 4,
    SPMV_GATHER_L1_TMA4 = 5,
    SPMV_GATHER_L1_TMA4_QUARTER = 6,
    SPMV_GATHER_TMA4_16 = 7,
    SPMV_GATHER_STREAM_LDG = 8,
    SPMV_GATHER_STREAM_BULK = 9,
    SPMV_GATHER_STREAM_CPASYNC = 10,
    SPMV_GATHER_STREAM_LDG_OCC = 11,
    SPMV_GATHER_STREAM_LDG_STS = 12,
    SPMV_GATHER_STREAM_LDG_FEW = 13,
    SPMV_GATHER_STREAM_LDG_RES_1 = 14, /* .. _RES_6 = 19 */
    SPMV_GATHER_STREAM_LDG_RES_6 = 19,
    SPMV_GATHER_TEX = 20               /* element fetches from a linear texture object over x (the call
                                          synchronises the stream: the object must outlive the launch) */
} spmv_gather_path_t;

spmv_status_t spmv_gather_ceiling(int32_t path, int32_t nnz, const int32_t *col_idx, int32_t n, const void *x,
                                  const void *vals, spmv_dtype_t dtype, uint64_t *checksum, int32_t *error,
                                  spmv_stream_t stream);

/*
 * Sparse times sparse, C = A * B, after OpSparse ("OpSparse: a highly
 * optimized framework for sparse general matrix multiplication on GPUs",
 * sections 3 and 5): Gustavson's row-by-row product (row i of C sums, over
 * the entries a_ip of row i of A, a_ip times row p of B), in two phases.
 *
 * spmv_spgemm_create takes the PATTERNS of A (m-by-k: a_row_ptr[m+1],
 * a_col_idx[a_nnz]) and B (k-by-n: b_row_ptr[k+1], b_col_idx[b_nnz]), device
 * int32 CSR arrays that the handle borrows until it is destroyed (their
 * contents must not change meanwhile).  It checks both as
 * spmv_plan_create does, counts the products of each row of C, bins the
 * rows by that count, sizes every row of C (the symbolic phase: sorted
 * lists for rows of at most 16 products, hash sets in shared memory up to
 * 4096; above, a dense row of C per row in global memory, the row's
 * products cut into equal pieces of at most 32768, a CTA each, with up to
 * 8 GiB of such rows at once),
 * and writes the number of entries of C to *c_nnz (HOST).  An entry of C
 * exists where at least one product lands, even if the products sum to
 * zero.  Synchronous (it waits for `stream` several times).
 * Limits: m, k, n >= 0; m + a_nnz and k + b_nnz < 2^31; C must have fewer
 * than 2^31 entries (else INVALID_ARG, with *c_nnz still set).
 * Errors: INVALID_ARG, INVALID_CSR, ALLOC, CUDA, UNSUPPORTED.  On error
 * *out is NULL.
 *
 * spmv_spgemm_compute is the numeric phase: with the values a_vals[a_nnz]
 * and b_vals[b_nnz] (device, the handle's value type) it writes C in CSR
 * form into caller-allocated device arrays c_row_ptr[m+1] (int32),
 * c_col_idx[c_nnz] (int32, increasing within each row) and c_vals[c_nnz].
 * It may be called again with new values of the same patterns.
 * Asynchronous on `stream`; allocates nothing.  Outside the rows of at
 * most 16 products (summed in the order of the row's products), the
 * products of an entry are added in an order that may change from call to
 * call (atomics), so its last bits may too; the pattern is always the same.
 * Errors: INVALID_ARG (null handle or pointers), CUDA.
 */
typedef struct spmv_spgemm_s *spmv_spgemm_t;

typedef struct {
    int32_t m, k, n;
    int32_t dtype;               /* spmv_dtype_t */
    int64_t a_nnz, b_nnz, c_nnz;
    int64_t products;            /* sum over the rows of C of their products */
    int64_t bin_rows[8];         /* rows of C by products: <= 16, <= 128, <= 512, <= 1024,
                                    <= 2048, <= 4096, more (the dense bin); [7] unused */
    int32_t dense_slots;         /* dense-bin rows of C held at once (one wave) */
    int32_t launches_per_compute;/* kernel launches one spmv_spgemm_compute issues */
    int64_t workspace_bytes;     /* device memory the handle owns */
    int64_t dense_pieces;        /* dense-bin pieces of at most 32768 products, a CTA each */
    int64_t dense_waves;         /* waves of dense-bin rows (two launches each) */
    int64_t numeric_bin_rows[8]; /* the numeric phase's bins: rows of at most 16 products,
                                    then by entries of C (<= 128, <= 512, <= 1024, <= 2048,
                                    <= 4096; tables of twice that), the dense bin as above */
} spmv_spgemm_info_t;

spmv_status_t spmv_spgemm_create(spmv_spgemm_t *out, int32_t m, int32_t k, int32_t n, int32_t a_nnz,
                                 const int32_t *a_row_ptr, const int32_t *a_col_idx, int32_t b_nnz,
                                 const int32_t *b_row_ptr, const int32_t *b_col_idx, spmv_dtype_t dtype,
                                 int64_t *c_nnz, spmv_stream_t stream);

spmv_status_t spmv_spgemm_compute(spmv_spgemm_t handle, const void *a_vals, const void *b_vals,
                                  int32_t *c_row_ptr, int32_t *c_col_idx, void *c_vals, spmv_stream_t stream);

/* Fill *info (HOST). */
spmv_status_t spmv_spgemm_info(spmv_spgemm_t handle, spmv_spgemm_info_t *info);

/* Kernel-side failure flags (HOST *flags; waits for the device).  Bit 1: a
 * row of C outgrew the size the symbolic phase found (the patterns changed
 * after creation); that row is incomplete. */
spmv_status_t spmv_spgemm_device_status(spmv_spgemm_t handle, int32_t *flags);

/* Free the handle's workspace (waits for the device).  NULL is a no-op. */
spmv_status_t spmv_spgemm_destroy(spmv_spgemm_t handle);

/*
 * Operators of language models whose data is ragged the way a sparse
 * matrix's rows are.  The pages have no counterpart.  In a decoder with
 * mixtures of experts two index structures decide what is read:
 *
 *   - the routing matrix R, tokens by experts with top_k entries per row:
 *     its transpose lists each expert's tokens (spmv_route_build: the
 *     tokens sorted by expert), R^T X gathers their rows
 *     (spmv_route_dispatch), and R weighted by the router, times the
 *     experts' rows, brings them back (spmv_route_combine);
 *   - the page table of a key-value cache, requests by pages, rows of one
 *     page to thousands: spmv_pages_append extends it and maps each new
 *     token to its slot, spmv_paged_store writes keys and values there, and
 *     spmv_paged_attention reduces each request's row of it.
 *
 * All of them are asynchronous on `stream`, allocate nothing and never
 * synchronise, so they can be captured in a CUDA graph; index arrays and
 * workspaces are the caller's (device).  Row strides (ld...) count
 * elements and may exceed the row's length, or be 0 or negative where
 * only reads use them.  Inputs and outputs must not overlap unless a
 * function says so.  Sums, dot products and softmax statistics are held in
 * 32 bits and rounded once; no result depends on the order in which blocks
 * run.
 */
typedef enum { SPMV_ELEM_F32 = 0, SPMV_ELEM_BF16 = 1, SPMV_ELEM_F16 = 2 } spmv_elem_t;

/* Bytes of workspace (HOST *bytes; 0 possible) spmv_route_build needs.  More
 * tokens never need less: a workspace for the most serves them all. */
spmv_status_t spmv_route_workspace(int32_t tokens, int32_t top_k, int32_t experts, size_t *bytes);

/*
 * Sort the entries of the routing matrix by expert.  Entry i = t * top_k + j
 * is token t's j-th choice, the expert expert_ids[t * ld_ids + j] (device,
 * int32 if id_bytes is 4, int64 if 8).  An id outside [0, experts) marks a
 * dropped entry (over an expert's capacity, held by another device, or
 * padding).  Writes
 *   expert_ptr[experts + 1]  row pointers: expert e owns the positions
 *                            expert_ptr[e] .. expert_ptr[e+1] - 1;
 *   entry[tokens * top_k]    the entry at each position, increasing within
 *                            an expert; the dropped entries, increasing,
 *                            fill the positions from expert_ptr[experts];
 *   slot[tokens * top_k]     the inverse: entry i's position p, or -1 - p
 *                            for a dropped entry.
 * Limits: tokens * top_k < 2^31, 1 <= experts <= 2048.  The workspace holds
 * at least spmv_route_workspace bytes, 16-byte aligned; its contents do not
 * matter.
 * Errors: INVALID_ARG, CUDA.
 */
spmv_status_t spmv_route_build(int32_t tokens, int32_t top_k, int32_t experts, const void *expert_ids,
                               int32_t id_bytes, int64_t ld_ids, int32_t *expert_ptr, int32_t *entry, int32_t *slot,
                               void *workspace, size_t workspace_bytes, spmv_stream_t stream);

/*
 * xs[p] = x[entry[p] / top_k] for every position p of the sorted order: x is
 * tokens-by-hidden, xs (tokens * top_k)-by-hidden, row-major.  Rows of
 * dropped entries (the last ones of xs) are set to zero, so xs is written
 * whole.  A copy: NaN payloads and signed zeros are kept.  The gradient of x
 * is spmv_route_combine of xs's gradient with null weights.
 * Limits, here and in the two functions below: tokens * top_k < 2^31, hidden <
 * 2^31 - 1024, tokens * hidden (rounded up to a multiple of 32) < 2^39.
 * Errors: INVALID_ARG, CUDA.  tokens, top_k or hidden of 0 is a no-op.
 */
spmv_status_t spmv_route_dispatch(int32_t tokens, int32_t top_k, int32_t hidden, spmv_elem_t elem,
                                  const int32_t *slot, const void *x, int64_t ldx, void *xs, int64_t ldxs,
                                  spmv_stream_t stream);

/*
 * y[t] = sum over j, in order, of weights[t * ldw + j] * ys[slot[t, j]]; a
 * dropped entry adds nothing, whatever its weight and row hold, and a token
 * with every entry dropped gets zeros.  weights is float32; null means 1.
 * Errors: as spmv_route_dispatch.  top_k of 0 sets y to zero.
 */
spmv_status_t spmv_route_combine(int32_t tokens, int32_t top_k, int32_t hidden, spmv_elem_t elem,
                                 const int32_t *slot, const float *weights, int64_t ldw, const void *ys,
                                 int64_t ldys, void *y, int64_t ldy, spmv_stream_t stream);

/*
 * The gradient of spmv_route_combine: from dy (tokens-by-hidden) and the
 * forward pass's ys and weights,
 *   dys[slot[t, j]] = weights[t, j] * dy[t]      (elem; null weights: dy[t])
 *   dweights[t * lddw + j] = <dy[t], ys[slot[t, j]]>   (float32)
 * Rows of dropped entries of dys and their dweights are set to zero.
 * dweights may be null (ys is then not read and may be null too).  dys may
 * be ys itself (the same pointer and row stride).
 * Errors: as spmv_route_dispatch.
 */
spmv_status_t spmv_route_combine_backward(int32_t tokens, int32_t top_k, int32_t hidden, spmv_elem_t elem,
                                          const int32_t *slot, const float *weights, int64_t ldw, const void *dy,
                                          int64_t lddy, const void *ys, int64_t ldys, void *dys, int64_t lddys,
                                          float *dweights, int64_t lddw, spmv_stream_t stream);

/* Bytes of workspace (HOST *bytes; 0 possible) spmv_pages_append needs. */
spmv_status_t spmv_pages_workspace(int32_t requests, size_t *bytes);

/*
 * Extend the page tables of a step's requests and map their new tokens to
 * cache slots.  Request r holds past[r] tokens, so the first
 * ceil(past[r] / page_size) entries of its table row (table + r * ld_table,
 * room for max_pages) are its pages; fresh[r] >= 0 tokens are added to it.
 * The pages they need beyond those held are taken from free_pages[num_free]
 * in its order, request by request, and written into the row.  Writes
 *   token_ptr[requests + 1]  prefix sums of fresh: request r's new tokens
 *                            are token_ptr[r] .. token_ptr[r+1] - 1;
 *   lens[requests]           past + fresh;
 *   positions[max_tokens]    each new token's position in its request;
 *   slots[max_tokens]        page * page_size + position % page_size;
 *   taken[1]                 how many of free_pages are used up (a prefix);
 *   status[1]                the flags below, OR-ed into what it holds.
 * Entries of slots and positions past the last new token are set to -1.  A
 * request that does not fit whole (the free list ends, the row would be
 * longer than max_pages, or its new tokens end past max_tokens) is not
 * served: its lens stays at past, its slots are -1 and its row is unchanged.
 * One that would outgrow its row takes no pages; the others still count in
 * the free list's order, so after one for which the list ends no later one
 * that needs pages is served.  Flags: bit 0 the free list ended; bit 1 a row
 * is too short; bit 2 more than max_tokens new tokens; bit 3 a negative past
 * or fresh (taken as 0), or a past beyond the row (that request is not
 * served); bit 4 a page outside [0, num_pages) among those used (its tokens'
 * slots are -1).
 * Limits: page_size >= 1, num_pages * page_size < 2^31, the sums of past and
 * fresh over the requests < 2^31.  past and fresh must not overlap an output (a
 * step's lens is copied before it is the next step's past).  The workspace holds at least
 * spmv_pages_workspace bytes, 16-byte aligned.
 * Errors: INVALID_ARG, CUDA.
 */
spmv_status_t spmv_pages_append(int32_t requests, const int32_t *past, const int32_t *fresh, int32_t page_size,
                                int32_t num_pages, const int32_t *free_pages, int32_t num_free, int32_t *table,
                                int64_t ld_table, int32_t max_pages, int32_t max_tokens, int32_t *token_ptr,
                                int32_t *lens, int32_t *slots, int32_t *positions, int32_t *taken, int32_t *status,
                                void *workspace, size_t workspace_bytes, spmv_stream_t stream);

/*
 * Write the keys and values of `tokens` new tokens into a paged cache: for
 * each i with slots[i] in [0, num_pages * page_size), page = slots[i] /
 * page_size, s = slots[i] % page_size, and every head h,
 *   k_cache[page * k_cache_stride[0] + s * k_cache_stride[1] + h * k_cache_stride[2] + d]
 *     = k[i * k_stride[0] + h * k_stride[1] + d],   0 <= d < head_dim,
 * and likewise v.  Other slots are skipped.  Strides (HOST arrays) count
 * elements; the last index is contiguous.  Two tokens must not share a slot.
 * Limits: num_pages * page_size < 2^31, heads * head_dim < 2^30, tokens *
 * heads * head_dim < 2^41.
 * Errors: INVALID_ARG, CUDA.
 */
spmv_status_t spmv_paged_store(int32_t tokens, int32_t heads, int32_t head_dim, spmv_elem_t elem,
                               const int32_t *slots, int32_t num_pages, int32_t page_size, const void *k,
                               const int64_t *k_stride, const void *v, const int64_t *v_stride, void *k_cache,
                               const int64_t *k_cache_stride, void *v_cache, const int64_t *v_cache_stride,
                               spmv_stream_t stream);

/*
 * Attention of one new token per request over a paged cache.  For request b
 * and query head h, with kv head c = h / (q_heads / kv_heads) and positions
 * t < lens[b], the key and value of position t in slot t % page_size of page
 * table[b * table_stride + t / page_size]:
 *   s_t = scale * <q[b, h], k_t>,   lse[b, h] = log sum_t exp(s_t),
 *   out[b, h] = sum_t exp(s_t - lse[b, h]) v_t.
 * A request of length 0 gets out = 0 and lse = -infinity.  Table entries past
 * a request's last page, and cache contents past its length, are not used
 * (they may hold anything, NaN included).  16-bit products are summed in 32
 * bits with weights of two elements each (16 or 22 bits; f16 weights in steps
 * of no less than 2^-39 of a row's largest).  An infinity in V makes its
 * element infinite, or NaN where its weight is lost (below 2^-126 of the row's
 * largest, f16 2^-40) or another infinity has the other sign; a score of minus
 * infinity weighs nothing, a row of such scores only gets out = 0 and lse =
 * -infinity, and a score of plus infinity or NaN makes its row NaN.
 *
 * The positions of all requests and kv heads together are cut into equal
 * shares, one per warp, whatever the lengths (the equal shares of the
 * merge-path SpMV); requests cut between warps and blocks are joined in a
 * fixed order, so results do not change from call to call.
 */
typedef struct {
    int32_t batch, q_heads, kv_heads, head_dim; /* q_heads a multiple of kv_heads; head_dim a
                                                   multiple of 8, at most 256; q_heads * head_dim
                                                   < 2^30 */
    int32_t page_size, num_pages, max_pages;    /* max_pages: entries in a table row */
    int32_t elem;                               /* spmv_elem_t of q, the caches and out */
    float scale;
    int32_t reserved;
    int64_t q_stride[2];   /* request, head (elements, as all strides) */
    int64_t k_stride[3];   /* page, position in it, head; multiples of 16 bytes */
    int64_t v_stride[3];
    int64_t out_stride[2]; /* request, head */
    int64_t table_stride;
    const void *q;
    const void *k_cache;   /* 16-byte aligned */
    const void *v_cache;
    const int32_t *table;
    const int32_t *lens;
    void *out;
    float *lse;            /* [batch * q_heads], or null */
    void *workspace;       /* spmv_paged_attention_workspace bytes, 16-byte aligned; the first 4096
                              are zeroed once by the caller, every call leaves them ready for the
                              next; calls that may overlap on the GPU need workspaces of their
                              own */
    size_t workspace_bytes;
    int32_t *status;       /* device int32; flags are OR-ed in.  Bit 0: a page outside
                              [0, num_pages) (its positions are left out); bit 1: a length that is
                              negative or longer than its row (taken as 0, or cut) */
} spmv_paged_attention_t;

/* Bytes of workspace (HOST *bytes) spmv_paged_attention needs for up to
 * max_batch requests, on the current device. */
spmv_status_t spmv_paged_attention_workspace(int32_t max_batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                             spmv_elem_t elem, size_t *bytes);

/* args is a HOST structure, read before the call returns.
 * Errors: INVALID_ARG, CUDA. */
spmv_status_t spmv_paged_attention(const spmv_paged_attention_t *args, spmv_stream_t stream);

/*
 * A paged cache of elements, or of 8-bit codes with scales.  Codes are e4m3:
 * a sign, four exponent and three mantissa bits, no infinities, largest value
 * 448, NaN 0x7f.  `block` neighbouring positions of a page share a float32
 * scale per head: page * page_size / block + s / block is the block of
 * position s of a page, and element d of it stands for
 *   value(k_cache[page * k_stride[0] + s * k_stride[1] + h * k_stride[2] + d])
 *     * k_scales[page * k_scale_stride[0] + (s / block) * k_scale_stride[1] + h * k_scale_stride[2]].
 */
typedef struct {
    int32_t num_pages, page_size; /* num_pages * page_size < 2^31 */
    int32_t block;                /* divides page_size; 0: the cache holds elements, no scales */
    int32_t reserved;
    int64_t k_stride[3];          /* page, position in it, head (elements or codes); the last index is contiguous */
    int64_t v_stride[3];
    int64_t k_scale_stride[3];    /* page, block in it, head */
    int64_t v_scale_stride[3];
    void *k_cache;
    void *v_cache;
    float *k_scales;
    float *v_scales;
} spmv_paged_cache_t;

/*
 * spmv_paged_store into a cache of codes (cache is a HOST structure, read
 * before the call returns, with 1 <= block <= 64).  For a block of positions
 * that tokens of this call are written to, a head, and keys or values:
 *   need = the least power of two p >= 2^-126 with every finite |x| <= 448 p,
 *          x over those tokens;
 *   old  = the scale held; where the block's first position is written, the
 *          block begins anew, and nothing it held counts;
 *   new  = need in a block that begins anew, else max(old, need).
 * The tokens' codes are x / new rounded to nearest, ties to even, NaN where x
 * is not finite; new is stored; and where new > old in a block that does not
 * begin anew the codes of its other positions become code * (old / new),
 * rounded (exact for powers of two, but for codes below 2^-6).  The codes of
 * the other positions of a block that begins anew stay as they are, without
 * meaning.  So a block filled from its first position on, in any number of
 * calls, keeps one scale for what it holds.
 * Tokens of one call that go to the same block are neighbours in slots, in any
 * order, skipped slots and at most 63 of these between two (as
 * spmv_pages_append places them); with block 1 any order will do.  Two tokens
 * must not share a slot.  Where either does not hold, what the blocks
 * concerned hold is not specified.
 * Limits: as spmv_paged_store, tokens * heads < 2^33, heads < 2^24.
 * Errors: INVALID_ARG, CUDA.
 */
spmv_status_t spmv_paged_store_e4m3(int32_t tokens, int32_t heads, int32_t head_dim, spmv_elem_t elem, const int32_t *slots,
                                    const spmv_paged_cache_t *cache, const void *k, const int64_t *k_stride, const void *v,
                                    const int64_t *v_stride, spmv_stream_t stream);

/*
 * Read requests' positions back from a paged cache into packed rows: row i of
 * k and v (i * k_stride[0] + h * k_stride[1] + d), token_ptr[r] <= i <
 * token_ptr[r + 1], is position i - token_ptr[r] of request r, whose pages are
 * row r of table (table + r * table_stride, max_pages entries).  token_ptr
 * (device, requests + 1) does not fall and begins at 0.  A cache of codes
 * gives code * scale in 32 bits, rounded to elem (block > 0); a cache of elements
 * (block 0, type elem) is copied.  Rows behind token_ptr[requests] or from
 * `tokens` on are left as they were; rows whose page is outside
 * [0, num_pages) or past max_pages are zeros.
 * Limits: tokens * heads * head_dim < 2^40, heads * head_dim < 2^30.
 * Errors: INVALID_ARG, CUDA.
 */
spmv_status_t spmv_paged_load(int32_t requests, int32_t tokens, int32_t heads, int32_t head_dim, spmv_elem_t elem,
                              const int32_t *table, int64_t table_stride, int32_t max_pages, const int32_t *token_ptr,
                              const spmv_paged_cache_t *cache, void *k, const int64_t *k_stride, void *v,
                              const int64_t *v_stride, spmv_stream_t stream);

/*
 * spmv_paged_attention over caches of codes: the key of position t is its
 * codes times its key scale, and likewise the value (spmv_paged_cache_t has
 * the layout; the scales are finite and positive, powers of two or not).  args->elem is the type
 * of q and out, bf16 or f16; k_cache and v_cache hold codes and their strides
 * count these (multiples of 16); head_dim is a multiple of 16.  q is taken in
 * f16 times a power of two per head, without loss down to 2^-29 of the head's
 * largest element; weights times value scales in 22 bits, in steps of no less
 * than 2^-38 of a row's largest weight times its largest value scale.  Dot
 * products, q times a key scale, and the sums of exp(s_t - max s) v_t have to
 * stay in the range of 32 bits.  A NaN
 * code of a position makes its score, or its element of the output, NaN.
 * workspace: spmv_paged_attention_e4m3_workspace bytes.  For the rest as
 * spmv_paged_attention.
 * Errors: INVALID_ARG, CUDA.
 */
spmv_status_t spmv_paged_attention_e4m3_workspace(int32_t max_batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                                  spmv_elem_t elem, size_t *bytes);
spmv_status_t spmv_paged_attention_e4m3(const spmv_paged_attention_t *args, int32_t block, const float *k_scales,
                                        const int64_t *k_scale_stride, const float *v_scales, const int64_t *v_scale_stride,
                                        spmv_stream_t stream);

/*
 * Attention of packed prompts, or of chunks of them behind what their
 * requests hold already.  Request r's queries are rows q_ptr[r] ..
 * q_ptr[r + 1] - 1 of q (nq of them), its keys and values rows kv_ptr[r] ..
 * kv_ptr[r + 1] - 1 of k and v (nk), kv head c = h / (q_heads / kv_heads) for
 * query head h.  Query i (0 <= i < nq) sees the keys j <= i + nk - nq where
 * `causal` is not 0 (its last query stands at its last key), else all:
 *   s_j = scale * <q_i, k_j>,   lse = log sum_j exp(s_j),
 *   out_i = sum_j exp(s_j - lse) v_j   over the keys it sees.
 * A query that sees none gets out = 0 and lse = -infinity.  Keys and values
 * that a query does not see may hold anything, NaN and infinities included;
 * rows of out and lse that belong to no request are left as they were.  Sums
 * and the softmax are in 32 bits; a weight is rounded to the elements' type
 * once, as the second product's operand.  The sums over keys are divided at
 * the end: exp(s_j - max s) v_j over a row's keys has to stay in the range of
 * 32 bits.  A score of minus infinity weighs nothing, a row of such scores only
 * gets out = 0 and lse = -infinity, and a score of plus infinity or NaN makes
 * its row NaN.  In other rows a value that is not finite counts however little
 * its key weighs: its element is that infinity, or NaN where the row sees a NaN
 * or infinities of both signs there (with a score of minus infinity it may
 * count or not).
 */
typedef struct {
    int32_t requests, tokens, keys; /* tokens: rows of q and out, keys: rows of k and v; each at most 2^31 - 513 */
    int32_t q_heads, kv_heads;      /* q_heads a multiple of kv_heads, at most 128 times as many;
                                       tokens * q_heads < 2^31 */
    int32_t head_dim;               /* a multiple of 8, at most 256 */
    int32_t elem;                   /* spmv_elem_t of q, k, v and out: bf16 or f16 */
    int32_t causal;
    float scale;
    int32_t reserved;
    int64_t q_stride[2];            /* row, head (elements); multiples of 16 bytes, as are the addresses;
                                       those of q, k and v are positive and less than 2^38.  Of a
                                       dimension of one element they are of no matter */
    int64_t k_stride[2];
    int64_t v_stride[2];
    int64_t out_stride[2];
    const void *q;
    const void *k;
    const void *v;
    const int32_t *q_ptr;           /* [requests + 1], device; do not fall */
    const int32_t *kv_ptr;          /* [requests + 1], or null: q_ptr */
    void *out;
    float *lse;                     /* [tokens * q_heads], or null */
    int32_t *status;                /* device int32; flags are OR-ed in.  Bit 0: a request's queries are
                                       not rows of q, bit 1: its keys are not rows of k; such a request
                                       is left out, its rows of out stay as they were.  Bit 2: a wait
                                       inside the kernel ran out (a second, and 256 clocks for each key
                                       and request of the call), and out is not complete */
    void *workspace;                /* spmv_prompt_attention_workspace bytes (fewer serve in part), 16-byte
                                       aligned, or null: where few queries leave SMs without work, their
                                       keys are cut into shares as far as it goes.  Its contents do not
                                       matter; calls that may overlap on the GPU need workspaces of their
                                       own */
    size_t workspace_bytes;
} spmv_prompt_attention_t;

/* Bytes of workspace (HOST *bytes) that spmv_prompt_attention has use for, on the current device. */
spmv_status_t spmv_prompt_attention_workspace(int32_t q_heads, int32_t kv_heads, int32_t head_dim, spmv_elem_t elem, size_t *bytes);

/* args is a HOST structure, read before the call returns.
 * Errors: INVALID_ARG, CUDA.  No requests, tokens or heads: nothing is done. */
spmv_status_t spmv_prompt_attention(const spmv_prompt_attention_t *args, spmv_stream_t stream);

/* Static text for a status code. */
const char *spmv_status_string(spmv_status_t status);

/* Description of the last error on the calling thread ("" if none). */
const char *spmv_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LBCSR_SPMV_H */
