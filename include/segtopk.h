/*
 * segtopk — segmented (batched) top-k by multi-pass radix digit selection,
 * written for NVIDIA GB300 (sm_103a).
 *
 * C ABI. All pointers are plain pointers; no C++ or framework types cross
 * this boundary. Every call is asynchronous on the given CUDA stream unless
 * its comment says otherwise.
 *
 * What is computed (per segment, independently):
 *   "Implement Segmented TopK using Thread-Block-Clusters" (CUB pull request),
 *   section 1 "High-level overview": for each of num_segments variable-length
 *   segments select the k largest (or smallest) keys, optionally carrying a
 *   value payload. The selection contract (which items, in which order) is
 *   the one of the CUB documentation page "Top-K: Determinism, Tie-Breaking,
 *   and Output Ordering" (sections "Requirements reference" and "Which items
 *   are selected?"), with +0.0 and -0.0 ranked as equal keys whose own bit
 *   patterns are written to the output ("Fix BlockTopK +/-0.0 handling",
 *   sections Cause and Fix).
 */
#ifndef SEGTOPK_H_
#define SEGTOPK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Exported entry points (the library is built with hidden visibility, so
 * that nothing else it contains can collide with another library's). */
#if defined(__GNUC__)
#define SEGTOPK_API __attribute__((visibility("default")))
#else
#define SEGTOPK_API
#endif

/* Key element types. Keys are read as raw bit patterns of this width. */
typedef enum {
  SEGTOPK_F16 = 0,  /* IEEE binary16 */
  SEGTOPK_BF16 = 1, /* bfloat16 */
  SEGTOPK_F32 = 2,  /* IEEE binary32 */
  SEGTOPK_F64 = 3,  /* IEEE binary64 */
  SEGTOPK_U32 = 4,  /* uint32_t */
  SEGTOPK_I32 = 5   /* int32_t */
} segtopk_dtype;

/* Which end of the order is selected (CUB's Max* / Min* entry points). */
typedef enum { SEGTOPK_MAX = 0, SEGTOPK_MIN = 1 } segtopk_direction;

/* Result-set reproducibility ("Top-K: Determinism, ...", "Determinism" table). */
typedef enum {
  SEGTOPK_NOT_GUARANTEED = 0,
  SEGTOPK_RUN_TO_RUN = 1,
  SEGTOPK_GPU_TO_GPU = 2
} segtopk_determinism;

/* Boundary tie policy (same page, "Tie-break" table). A concrete tie-break
 * requires SEGTOPK_GPU_TO_GPU. UNSPECIFIED is resolved as
 * PREFER_SMALLER_INDEX under RUN_TO_RUN and GPU_TO_GPU; under
 * NOT_GUARANTEED, boundary ties beyond those needed are taken in whatever
 * order the kernel meets them (any subset of the ties is a valid result). */
typedef enum {
  SEGTOPK_TIE_UNSPECIFIED = 0,
  SEGTOPK_PREFER_SMALLER_INDEX = 1,
  SEGTOPK_PREFER_LARGER_INDEX = 2
} segtopk_tie_break;

/* Output order of the selected items (same page, "Output ordering" table).
 * UNSORTED: any order; with a deterministic mode the set is fixed but the
 *         positions may differ from run to run (set membership, not
 *         positions, is what determinism pins).
 * SORTED: by key, better first; equal keys in unspecified order (this
 *         library sorts 64-bit keys on the key alone; single-warp paths
 *         with larger indices preferred write equal keys by descending
 *         index; otherwise equal keys come out in source-index order).
 * STABLE_SORTED: by key, better first; equal keys by source index ascending,
 *         whatever the tie-break. */
typedef enum {
  SEGTOPK_UNSORTED = 0,
  SEGTOPK_SORTED = 1,
  SEGTOPK_STABLE_SORTED = 2
} segtopk_ordering;

/* Status codes returned by every entry point. */
typedef enum {
  SEGTOPK_SUCCESS = 0,
  SEGTOPK_ERROR_INVALID_VALUE = 1,       /* bad enum, null pointer, negative size, k < 0 */
  SEGTOPK_ERROR_INVALID_COMBINATION = 2, /* determinism / tie_break pair not allowed */
  SEGTOPK_ERROR_NOT_SUPPORTED = 3,       /* size or k outside this library's limits */
  SEGTOPK_ERROR_MISALIGNED = 4,          /* a pointer not aligned to its element size */
  SEGTOPK_ERROR_CUDA = 5,                /* a CUDA runtime call failed: see segtopk_last_cuda_error */
  SEGTOPK_ERROR_DEVICE = 6               /* current device is not an sm_103 GPU */
} segtopk_status;

/* Largest k this library serves (the selected items of one segment are held
 * and sorted on chip). Calls with a larger k return SEGTOPK_ERROR_NOT_SUPPORTED. */
#define SEGTOPK_MAX_K 2048

/* Largest segment length (keys) accepted: segment-local indices are 32-bit. */
#define SEGTOPK_MAX_SEGMENT_LEN 2147483647LL

/*
 * Segmented top-k.
 *
 * Semantics: "Implement Segmented TopK using Thread-Block-Clusters", sections
 * 1.2 "Radix (digit) top-k" (method), 1.5 "Final filter and output placement"
 * and 1.6 "Determinism / tie-breaking"; contract of "Top-K: Determinism,
 * Tie-Breaking, and Output Ordering"; +/-0.0 handling of "Fix BlockTopK
 * +/-0.0 handling".
 *
 * Arguments (all device pointers unless stated):
 *   key_dtype        element type of keys and out_keys.
 *   keys             key array; segment s covers elements
 *                    [segment_offsets[s], segment_offsets[s+1]). Must be
 *                    aligned to its element size (any element of a larger
 *                    array may start it). Read only.
 *   values           optional int32 payload parallel to keys (NULL: keys only).
 *   segment_offsets  int64 array of num_segments + 1 element offsets, each
 *                    non-negative and within the key array. A segment whose
 *                    end is not greater than its begin is empty.
 *   num_segments     number of segments (>= 0).
 *   k                items to select per segment (>= 0).
 *   direction, determinism, tie_break, ordering: see the enums. Valid
 *                    (determinism, tie_break) pairs: (any, UNSPECIFIED) and
 *                    (GPU_TO_GPU, PREFER_SMALLER_INDEX | PREFER_LARGER_INDEX).
 *   out_keys         num_segments * k elements; segment s writes slots
 *                    [s*k, s*k + min(k, n_s)) with the original key bits and
 *                    leaves [s*k + n_s, s*k + k) untouched when n_s < k.
 *   out_values       num_segments * k int32; required iff values != NULL;
 *                    out_values[j] = values[segment_offsets[s] + i] for the
 *                    element i written to out_keys[j].
 *   max_segment_len  host-side upper bound on every segment's length. A
 *                    negative value means unknown: the library then copies
 *                    segment_offsets to the host and waits for the stream
 *                    (a synchronising call). A bound that is too small is a
 *                    caller error: longer segments are left unwritten.
 *   stream           cudaStream_t (NULL = the legacy default stream).
 *
 * Ownership: the caller owns every buffer. The library allocates no device
 * memory; it caches device attributes and per-kernel shared-memory limits.
 * Inputs must not overlap outputs.
 *
 * Errors: argument errors are detected on the host before any launch and
 * nothing is launched. num_segments == 0 or k == 0 is a successful no-op.
 * A failed launch returns SEGTOPK_ERROR_CUDA (segtopk_last_cuda_error()
 * gives the cudaError_t). The call does not synchronise (except as noted
 * for max_segment_len < 0).
 */
SEGTOPK_API int segtopk_batched_topk(segtopk_dtype key_dtype, const void* keys, const int32_t* values,
                         const int64_t* segment_offsets, int64_t num_segments, int32_t k,
                         segtopk_direction direction, segtopk_determinism determinism,
                         segtopk_tie_break tie_break, segtopk_ordering ordering, void* out_keys,
                         int32_t* out_values, int64_t max_segment_len, void* stream);

/* Optional launch controls for segtopk_batched_topk_ex (zero = automatic). */
typedef struct {
  /* CTAs per segment: 0 chooses it from the occupancy the device reports
   * (fewest waves, ties toward the widest cluster); 1..16 forces the width
   * (widths above 8 need non-portable cluster support). */
  int32_t cluster_width;
  /* Warp-select paths (used when k <= 32): segments of at most
   * small_segment_max_len keys take one warp each, longer ones of at most
   * team_segment_max_len keys a team of eight warps each; longer segments
   * (and every segment when k > 32) take one CTA or cluster each. 0 chooses
   * the defaults below (none when cluster_width is forced); a negative value
   * turns that path off. */
  int32_t small_segment_max_len;
  int32_t team_segment_max_len;
  int32_t reserved[5]; /* must be zero */
} segtopk_options;

/* Default limits of the warp-select paths. With at least as many segments as
 * SMs: one warp per segment up to SEGTOPK_SMALL_SEGMENT_DEFAULT keys and no
 * team range (SEGTOPK_TEAM_SEGMENT_DEFAULT does not exceed it: longer
 * segments are faster on the CTA path then). With fewer segments: no
 * single-warp range and teams of eight warps up to SEGTOPK_TEAM_SEGMENT_FEW
 * keys. */
#define SEGTOPK_SMALL_SEGMENT_DEFAULT 4096
#define SEGTOPK_TEAM_SEGMENT_DEFAULT 4096
#define SEGTOPK_TEAM_SEGMENT_FEW 8192

/* segtopk_batched_topk with launch controls; options may be NULL. Returns
 * SEGTOPK_ERROR_INVALID_VALUE for a width outside 0..16 or nonzero reserved
 * fields, and SEGTOPK_ERROR_NOT_SUPPORTED when the device cannot launch the
 * requested width. Without options (and in segtopk_batched_topk), the
 * warp-select paths take the segments their default limits give when
 * k <= 32; the others take one CTA or cluster each. */
SEGTOPK_API int segtopk_batched_topk_ex(segtopk_dtype key_dtype, const void* keys, const int32_t* values,
                            const int64_t* segment_offsets, int64_t num_segments, int32_t k,
                            segtopk_direction direction, segtopk_determinism determinism,
                            segtopk_tie_break tie_break, segtopk_ordering ordering, void* out_keys,
                            int32_t* out_values, int64_t max_segment_len,
                            const segtopk_options* options, void* stream);

/*
 * segtopk_batched_topk_ex with a payload of 4- or 8-byte values: values and
 * out_values point to value_bytes-wide elements (int32_t or int64_t; any
 * 8-byte payload, such as a global index or a pointer, is copied as is).
 * value_bytes must be 4 or 8 when values is not NULL (else
 * SEGTOPK_ERROR_INVALID_VALUE). Everything else is as in
 * segtopk_batched_topk_ex; keys only when values and out_values are NULL.
 * (The pages' CUB pull request lists wider value types and larger segments
 * among its future work: "Implement Segmented TopK using
 * Thread-Block-Clusters", section 10 "Known limitations and future work".)
 */
SEGTOPK_API int segtopk_batched_topk_values(segtopk_dtype key_dtype, const void* keys, const void* values,
                                            int32_t value_bytes, const int64_t* segment_offsets,
                                            int64_t num_segments, int32_t k, segtopk_direction direction,
                                            segtopk_determinism determinism, segtopk_tie_break tie_break,
                                            segtopk_ordering ordering, void* out_keys, void* out_values,
                                            int64_t max_segment_len, const segtopk_options* options,
                                            void* stream);

/*
 * Top-k over one array (no segments): the k best of keys[0, num_keys),
 * with the same contract per mode as one segment of segtopk_batched_topk
 * (source index = array index). The CUB pull request's overview names this
 * operation (cub::DeviceTopK) beside the segmented one ("Implement Segmented
 * TopK using Thread-Block-Clusters", section 1.1).
 *
 * Method: two passes of the segmented selection. The array is split into P
 * balanced contiguous pieces (P = min(304, num_keys / max(65536, 16 k)), at
 * least 1); pass 1 writes each piece's k best, in stable sorted order, to the
 * workspace; pass 2 selects the k best of the P * k candidates. Pieces keep
 * source order and each piece's equal keys keep index order, so a
 * candidate's position orders ties as its array index does: tie-breaks and
 * stable order are exact.
 *
 * Arguments: keys, values, out_keys, out_values, workspace are device
 * pointers. values / out_values: optional payload of value_bytes (4 or 8)
 * per element, both NULL for keys only. out_keys / out_values hold k slots;
 * with num_keys < k only the first num_keys are written. workspace: at
 * least segtopk_topk_workspace_bytes(...) bytes, 256-byte aligned, owned by
 * the caller (the library allocates nothing). num_keys may exceed 2^31 as
 * long as every piece holds fewer than 2^31 keys.
 *
 * Errors as segtopk_batched_topk; a workspace that is too small returns
 * SEGTOPK_ERROR_INVALID_VALUE. Asynchronous on `stream` (up to three kernel
 * launches: the piece offsets, pass 1, pass 2).
 */
SEGTOPK_API size_t segtopk_topk_workspace_bytes(segtopk_dtype key_dtype, int32_t value_bytes, int64_t num_keys,
                                                int32_t k);
SEGTOPK_API int segtopk_topk(segtopk_dtype key_dtype, const void* keys, const void* values, int32_t value_bytes,
                             int64_t num_keys, int32_t k, segtopk_direction direction,
                             segtopk_determinism determinism, segtopk_tie_break tie_break,
                             segtopk_ordering ordering, void* out_keys, void* out_values, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * Same operation with HOST buffers: keys, values, segment_offsets, out_keys
 * and out_values are host pointers (pinned memory gives full copy
 * bandwidth). The caller also passes a device workspace of at least
 * segtopk_host_workspace_bytes(...) bytes, 256-byte aligned (the library
 * allocates nothing). The call copies the keys, the offsets and the output
 * slots to the device, runs the selection on `stream` (for pairs the kernel
 * writes each selected element's source index), copies the results back,
 * waits for the stream, and then gathers the selected values from the
 * caller's host `values` array, so that only the keys cross to the device.
 * The host outputs are ready on return.
 *
 * The host offsets are read on the host: every offset must be non-negative
 * (SEGTOPK_ERROR_INVALID_VALUE otherwise, before anything is copied or
 * launched), and max_segment_len is ignored (the true longest segment is
 * known). Slots past a short segment's length keep their host contents.
 */
SEGTOPK_API int segtopk_batched_topk_host(segtopk_dtype key_dtype, const void* keys, const int32_t* values,
                              const int64_t* segment_offsets, int64_t num_segments, int32_t k,
                              segtopk_direction direction, segtopk_determinism determinism,
                              segtopk_tie_break tie_break, segtopk_ordering ordering,
                              void* out_keys, int32_t* out_values, int64_t max_segment_len,
                              void* device_workspace, size_t workspace_bytes, void* stream);

/*
 * Size of the fixed device staging area of segtopk_batched_topk_host_noalloc:
 * 32 MiB. A request fits when segtopk_host_workspace_bytes(...) for its
 * sizes is at most this (for example about 8 million fp32 keys, with or
 * without int32 values: values stay on the host).
 */
#define SEGTOPK_NOALLOC_STAGING_BYTES (32u * 1024u * 1024u)

/*
 * segtopk_batched_topk_host for callers that cannot allocate device memory:
 * a plugin or library routine running inside a host program that owns the
 * GPU's memory (a framework whose caching allocator has reserved it, so that
 * a cudaMalloc of the caller's own would fail or fragment that pool), or
 * code held to a fixed device-memory budget with no per-call allocations.
 * The source pages have no counterpart of this entry point.
 *
 * Arguments, semantics and results are those of segtopk_batched_topk_host,
 * without the workspace: the device staging comes from a fixed array of
 * SEGTOPK_NOALLOC_STAGING_BYTES inside the library. Every GPU on which the
 * library's device code is loaded holds that array until the process exits.
 * The call runs on the current device, which must be the device of `stream`.
 *
 * Set-up: the first call on a device (with that device current) looks up the
 * array's device address once; make that first call before any stream
 * capture begins on the device. The address is kept for the life of the
 * process: a device reset (cudaDeviceReset) between calls is not supported.
 *
 * Limits and errors: a request needing more than SEGTOPK_NOALLOC_STAGING_BYTES
 * of staging returns SEGTOPK_ERROR_NOT_SUPPORTED before anything is copied.
 * Otherwise the status codes are those of segtopk_batched_topk_host. The call
 * makes no device allocation and frees nothing.
 *
 * Sharing: every call on a device uses the same array, which keeps the last
 * call's data; each call writes every byte it reads from it, so nothing needs
 * clearing. Calls whose GPU work overlaps (calls from several host threads,
 * or on several streams of one device) race on the array: serialise them.
 * Like segtopk_batched_topk_host, the call waits for `stream` before it
 * returns.
 */
SEGTOPK_API int segtopk_batched_topk_host_noalloc(segtopk_dtype key_dtype, const void* keys, const int32_t* values,
                                      const int64_t* segment_offsets, int64_t num_segments, int32_t k,
                                      segtopk_direction direction, segtopk_determinism determinism,
                                      segtopk_tie_break tie_break, segtopk_ordering ordering,
                                      void* out_keys, int32_t* out_values, int64_t max_segment_len,
                                      void* stream);

/* Device workspace bytes segtopk_batched_topk_host needs for these sizes
 * (num_keys = number of key elements the offsets address, i.e. the largest
 * segment end): keys, offsets, output keys and, for pairs, the selected
 * source indices. Host-only arithmetic; 0 for negative or oversized
 * arguments. */
SEGTOPK_API size_t segtopk_host_workspace_bytes(segtopk_dtype key_dtype, int has_values, int64_t num_keys,
                                    int64_t num_segments, int32_t k);

/* Human-readable text of a status code (static storage). */
SEGTOPK_API const char* segtopk_status_string(int status);

/* cudaError_t of the last SEGTOPK_ERROR_CUDA on the calling thread (0 if none). */
SEGTOPK_API int segtopk_last_cuda_error(void);

/*
 * Reads and clears the device-side error word of the current device. The
 * kernels bound every wait on an asynchronous copy; a wait that gives up
 * sets this word (bit 0: copy wait timed out; bit 1: a segment longer than
 * the launch was planned for; bit 2: an expert or token id past the last
 * one, see SEGTOPK_DEVICE_ERROR_INDEX). Synchronises the device. Returns a status;
 * the word is stored in *error_word.
 */
SEGTOPK_API int segtopk_read_device_error(uint32_t* error_word);

/* Number of kernel launches the last successful call on this thread made. */
SEGTOPK_API int segtopk_last_launch_count(void);

/*
 * Diagnostics of the instrumented build (the library compiled with
 * SEGTOPK_STATS and SEGTOPK_TEST_HOOKS, a separate shared object); the
 * ordinary build returns SEGTOPK_ERROR_NOT_SUPPORTED from both and changes
 * nothing. The source pages have no counterpart of either.
 *
 * segtopk_read_stats: synchronises the device, then sums and clears the
 * per-CTA counters of the segment kernel over every launch since the last
 * read: out[0] CTAs, [1] cycles, [2] cycles to the first bound, [3] cycles
 * of the stream (first bound included), [4] cycles after it (final
 * selection, merge, output), [5] ring chunks, [6] list trims, [7] slices
 * read twice, [8] list entries at the end of the stream, [9] slices with a
 * sampled first bound, [10] digit-selection passes, [11] cycles warp 0
 * waited for copies, [12] keys, [13] chunk shares of warp 0 that held
 * candidates, [14] chunk offers that overflowed the list, [15] - [17]
 * cycles of the small sampled bound's per-warp minimums, merge and write,
 * [18] / [19] cycles of a lone CTA's final selection and of its output,
 * [20] - [22] cycles of every block selection's digit passes, counting
 * finishes and compactions; n entries are written (zeros past 23).
 *
 * segtopk_set_test_hooks: the bound (SM clock cycles) after which a wait on
 * a bulk copy gives up, and a number of bytes (a multiple of 16, at most
 * 4096) added to the expected byte count of every slice's first copy, so
 * that its wait runs out: tests of the bounded wait use it. The kernel then
 * sets bit 0 of the device error word, writes no output for the affected
 * segments and returns.
 */
SEGTOPK_API int segtopk_read_stats(uint64_t* out, int n);
SEGTOPK_API int segtopk_set_test_hooks(long long wait_limit_cycles, uint32_t first_copy_extra_bytes);

/*
 * segtopk_test_device_prep (instrumented build; host only, no CUDA call):
 * replays the per-device launch-preparation decisions the library makes
 * before every launch, on fresh records, for n launches on device ordinals
 * devices[i]. A launch of the segment kernel has cluster_widths[i] >= 1 and
 * smem_bytes[i] of dynamic shared memory; cluster_widths[i] <= 0 denotes a
 * warp-kernel launch. actions[i] receives the attribute calls that launch
 * would make, every earlier one taken to have succeeded: bit 0 raises the
 * shared-memory opt-in, bit 1 allows clusters wider than 8, bit 2 sets the
 * warp kernel's carveout; ~0 for a device ordinal outside 0..63. Function
 * attributes belong to each device's copy of a kernel, so each device gets
 * its own calls. Errors: SEGTOPK_ERROR_INVALID_VALUE for n < 0 or a null
 * array with n > 0.
 */
SEGTOPK_API int segtopk_test_device_prep(int n, const int* devices, const uint32_t* smem_bytes,
                                         const int* cluster_widths, uint32_t* actions);

/*
 * ---------------------------------------------------------------------------
 * Row operators: expert routing, tokens sorted by expert and back, embedding
 * ---------------------------------------------------------------------------
 * The selection's neighbours in a model (the source pages have no counterpart):
 * the k best experts of every token with their weights; the tokens' rows in
 * the order of their experts and, weighted, back; the rows of a token
 * embedding; and the gradients of all three (the experts' products, layer norm
 * and rows in 8 bits follow below). Sorting is stable and there are
 * no atomics on results, so every result is the same from run to run.
 *
 * Common to all: device pointers unless stated; float types are F16, BF16 and
 * F32 (others: SEGTOPK_ERROR_NOT_SUPPORTED); sums are held in 32 bits and
 * rounded once, when they are written. A stride counts elements from one row
 * to the next, is not negative, and may be smaller than the width for inputs
 * (0: the same row for all); rows themselves are contiguous, and outputs are
 * dense. Pointers need the alignment of their elements; rows that start on
 * 16-byte boundaries and hold a multiple of 16 bytes move fastest. Calls are
 * asynchronous on `stream`, allocate nothing, may be captured in a graph, and
 * check their arguments before any launch. Outputs must not overlap inputs.
 */

/* Bit of the device error word (segtopk_read_device_error): an expert id not
 * below num_experts or a token not below the table's rows. Such an id counts
 * as none, like a negative one; negative ids are legitimate and set nothing. */
#define SEGTOPK_DEVICE_ERROR_INDEX 4u

/* Largest number of experts, and of experts chosen by segtopk_route. */
#define SEGTOPK_MAX_EXPERTS 1024
#define SEGTOPK_ROUTE_MAX_K 32

/* Scores of a token's experts. */
typedef enum {
  SEGTOPK_SOFTMAX = 0, /* exp(l_e - max) / sum over all experts */
  SEGTOPK_SIGMOID = 1  /* 1 / (1 + exp(-l_e)) */
} segtopk_score;

/*
 * The k best experts of each token, best first, and their weights.
 *
 * Chosen by score + bias (bias: `experts` float values, or NULL: none), ties
 * to the lower expert. The scores and sums are those of 32 bits, so two that
 * are less than their roundings apart may tie or change places; equal logits
 * with equal biases always tie. Without a bias the logits are compared, which
 * order as the scores do; +0.0 and -0.0 are equal, and NaN ranks above +inf.
 * Weights: scale * score, or with renormalize (0 or 1) scale * score / (sum
 * of the k chosen scores). The bias chooses only and is in no weight.
 *
 * An expert whose logit is -inf (or whose bias is) is never chosen: where
 * fewer than k are left, the last places get expert id -1 and weight 0. NaN
 * or +inf logits give the weights that the formula gives (NaN).
 *
 * logits: tokens rows of `experts` values of `dtype`, row_stride apart.
 * expert_ids, weights: tokens x k. Limits: 1 <= k <= experts, experts <=
 * SEGTOPK_MAX_EXPERTS, k <= SEGTOPK_ROUTE_MAX_K, tokens * k < 2^31.
 */
SEGTOPK_API int segtopk_route(segtopk_dtype dtype, const void* logits, int64_t tokens, int32_t experts,
                              int64_t row_stride, int32_t k, segtopk_score score, int renormalize, float scale,
                              const float* bias, int32_t* expert_ids, float* weights, void* stream);

/*
 * The same choice limited to groups of experts: the experts are num_groups
 * groups of equal size, in order; the groups_kept best groups are taken, and
 * in them the k best experts. A group's score is its best expert's
 * (SEGTOPK_GROUP_BEST), or the sum of its two best ones' score + bias
 * (SEGTOPK_GROUP_BEST_TWO; an expert that is never chosen adds nothing). Ties
 * go to the lower group. Weights, the softmax's sum among them, are over all
 * experts as above, and so is the gradient (segtopk_route_backward). With
 * SEGTOPK_GROUP_BEST and no bias the logits are compared, else scores of 32
 * bits. 1 <= groups_kept <= num_groups <= SEGTOPK_MAX_GROUPS, experts a
 * multiple of num_groups, k at most the experts of groups_kept groups.
 */
#define SEGTOPK_MAX_GROUPS 32
typedef enum { SEGTOPK_GROUP_BEST = 0, SEGTOPK_GROUP_BEST_TWO = 1 } segtopk_group_score;
SEGTOPK_API int segtopk_route_groups(segtopk_dtype dtype, const void* logits, int64_t tokens, int32_t experts,
                                     int64_t row_stride, int32_t k, int32_t num_groups, int32_t groups_kept,
                                     segtopk_group_score group_score, segtopk_score score, int renormalize,
                                     float scale, const float* bias, int32_t* expert_ids, float* weights,
                                     void* stream);

/*
 * Gradient of the logits from that of the weights (tokens x k): dense,
 * tokens x experts of `dtype`. expert_ids are the ones segtopk_route chose
 * (distinct per token; those outside 0 .. experts - 1 contribute nothing, as
 * if their weight were not there); score, renormalize and scale as there.
 */
SEGTOPK_API int segtopk_route_backward(segtopk_dtype dtype, const float* grad_weights, const void* logits,
                                       int64_t tokens, int32_t experts, int64_t row_stride, int32_t k,
                                       const int32_t* expert_ids, segtopk_score score, int renormalize,
                                       float scale, void* grad_logits, void* stream);

/*
 * Sorts token slots by expert, stably. expert_ids: `slots` ids (tokens x k,
 * in that order) of id_bytes 4 (int32) or 8 (int64); a negative one marks a
 * slot without an expert. Writes
 *   offsets      experts + 1 int64: expert e has the sorted rows
 *                [offsets[e], offsets[e + 1]) (usable as segment_offsets);
 *   row_of_slot  slots int32: the sorted row of each slot, or -1 for none;
 *   slot_of_row  slots int32: the slot of each sorted row; -1 from row
 *                offsets[experts] on.
 * workspace: at least segtopk_group_workspace_bytes(slots, experts) bytes
 * (which may be 0; host-only arithmetic), 4-byte aligned. experts <=
 * SEGTOPK_MAX_EXPERTS, slots < 2^31.
 */
SEGTOPK_API size_t segtopk_group_workspace_bytes(int64_t slots, int32_t experts);
SEGTOPK_API int segtopk_group(const void* expert_ids, int32_t id_bytes, int64_t slots, int32_t experts,
                              int64_t* offsets, int32_t* row_of_slot, int32_t* slot_of_row, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Copies the tokens' rows into sorted order: rows[r] = x[t] for the row r of
 * each of token t's k slots. Elements of 1, 2, 4 or 8 bytes are moved as they
 * are. rows: tokens * k dense rows; from row kept[0] (the last of
 * segtopk_group's offsets) on they are zeros.
 */
SEGTOPK_API int segtopk_dispatch(const void* x, int32_t element_bytes, int64_t tokens, int32_t k, int64_t width,
                                 int64_t x_stride, const int32_t* row_of_slot, const int64_t* kept, void* rows,
                                 void* stream);

/*
 * out[t] = sum over the slots j of token t that have a row r of weights[t, j]
 * * rows[r], in the order of the slots; weights (tokens x k) NULL: all 1,
 * which is the gradient of segtopk_dispatch. A token without a row gets
 * zeros, and rows that no slot has are not read.
 */
SEGTOPK_API int segtopk_combine(segtopk_dtype dtype, const void* rows, int64_t tokens, int32_t k, int64_t width,
                                int64_t row_stride, const int32_t* row_of_slot, const float* weights, void* out,
                                void* stream);

/*
 * Gradients of segtopk_combine with weights: grad_rows[r] = weights[t, j] *
 * grad_out[t] (tokens * k dense rows, zeros from kept[0] on) and
 * grad_weights[t, j] = the product of rows[r] and grad_out[t] (0 for a slot
 * without a row).
 */
SEGTOPK_API int segtopk_combine_backward(segtopk_dtype dtype, const void* grad_out, int64_t grad_stride,
                                         const void* rows, int64_t row_stride, int64_t tokens, int32_t k,
                                         int64_t width, const int32_t* row_of_slot, const int64_t* kept,
                                         const float* weights, void* grad_rows, float* grad_weights, void* stream);

/*
 * Embedding: out[i] = scale * table[tokens[i]], computed in 32 bits and
 * written as out_dtype. table: vocab rows of `width` values, row_stride
 * apart; tokens: num_tokens ids of token_bytes 4 (int32) or 8 (int64). A
 * token outside the table gives a row of zeros (a negative one on purpose,
 * as in a shard of a vocabulary; one past the last row also sets the device
 * error word). width <= 2^20, vocab < 2^31 - 1, num_tokens < 2^31.
 */
SEGTOPK_API int segtopk_embedding(segtopk_dtype dtype, const void* table, int64_t vocab, int64_t width,
                                  int64_t row_stride, const void* tokens, int32_t token_bytes, int64_t num_tokens,
                                  float scale, segtopk_dtype out_dtype, void* out, void* stream);

/*
 * Gradient of the table: grad_table[v] = scale * (sum of grad_out[i] over the
 * i with tokens[i] = v, in the order of i), as table_dtype; rows without a
 * token are zeros. With accumulate (0 or 1) that sum is added to grad_table
 * instead, and only the rows of tokens in the batch are read and written.
 * padding_token: a token that gets no gradient, or negative for none; tokens
 * outside the table get none either.
 *
 * workspace: at least segtopk_embedding_backward_workspace_bytes(...) bytes,
 * 256-byte aligned (host-only arithmetic; 0 for sizes out of range).
 */
SEGTOPK_API size_t segtopk_embedding_backward_workspace_bytes(int64_t num_tokens, int64_t vocab, int64_t width);
SEGTOPK_API int segtopk_embedding_backward(segtopk_dtype dtype, const void* grad_out, int64_t grad_stride,
                                           const void* tokens, int32_t token_bytes, int64_t num_tokens,
                                           int64_t vocab, int64_t width, int64_t padding_token, float scale,
                                           segtopk_dtype table_dtype, void* grad_table, int accumulate,
                                           void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The experts' products
 * ---------------------------------------------------------------------------
 * Between segtopk_dispatch and segtopk_combine: expert e's matrix product of
 * its rows [offsets[e], offsets[e + 1]), as segtopk_group sorted them
 * (offsets: experts + 1 int64 on the device, which the host does not read).
 * Rows of `rows` from offsets[experts] on, and before offsets[0] where that is
 * not 0, belong to no expert: they are not read into any result, and their rows
 * of `out` are zeros. An offset that is negative, past the rows or below an
 * earlier one counts as the nearest that is not.
 *
 * On the tensor cores: sums are held in 32 bits there, in an order that
 * depends on the sizes alone, and rounded once, to out_dtype (F16, BF16 or
 * F32). What TMA reads has 16-byte addresses and strides of a multiple of 16
 * bytes (else SEGTOPK_ERROR_MISALIGNED); strides of `rows` are at least their
 * width. Widths of up to 2^20, fewer than 2^31 - 256 rows, experts <=
 * SEGTOPK_MAX_EXPERTS; one launch a call, no workspace.
 */

/*
 * out[r, n] = sum_k rows[r, k] * weights[e, n, k], rows and weights of dtype
 * F16 or BF16, width (the number of k) a multiple of 8. weights: experts
 * matrices expert_stride apart; one of out_stride (between values of n) and
 * in_stride (of k) is 1 and the other at least the number of values of the
 * first, so that weights can be read transposed, as the rows' gradient does:
 * it is this product of out's gradient with n and k exchanged. With in_stride
 * other than 1 out_width is a multiple of 8. out: num_rows x out_width, dense.
 */
SEGTOPK_API int segtopk_expert_matmul(segtopk_dtype dtype, const void* rows, int64_t num_rows, int64_t width,
                                      int64_t row_stride, const void* weights, int32_t experts, int64_t out_width,
                                      int64_t expert_stride, int64_t out_stride, int64_t in_stride,
                                      const int64_t* offsets, segtopk_dtype out_dtype, void* out, void* stream);

/*
 * The same of rows and weights in 8 bits (e4m3: 1 sign, 4 exponent and 3
 * fraction bits, no infinities), each with a float scale for a block:
 *   out[r, n] = sum_b row_scales[r, b] * weight_scales[e, n / 128, b]
 *               * sum_{k of block b} rows[r, k] * weights[e, n, k]
 * with blocks b of 128 values of k, the last one in part where width is no
 * multiple of 128. width is a multiple of 16. row_scales: num_rows rows of
 * ceil(width / 128), scale_stride apart (segtopk_quantize_rows makes them);
 * weight_scales: experts x ceil(out_width / 128) x ceil(width / 128), dense.
 */
SEGTOPK_API int segtopk_expert_matmul_f8(const void* rows, int64_t num_rows, int64_t width, int64_t row_stride,
                                         const float* row_scales, int64_t scale_stride, const void* weights,
                                         int32_t experts, int64_t out_width, int64_t expert_stride,
                                         int64_t out_stride, const float* weight_scales, const int64_t* offsets,
                                         segtopk_dtype out_dtype, void* out, void* stream);

/*
 * The weights' gradient of segtopk_expert_matmul:
 *   out[e, a, b] = sum over expert e's rows r of a_rows[r, a] * b_rows[r, b],
 * experts x a_width x b_width, dense; zeros for an expert without rows. With
 * out's gradient as a and the rows as b it has the layout of weights whose k
 * is dense, and the other way round that of weights whose n is. Both widths
 * are multiples of 8.
 */
SEGTOPK_API int segtopk_expert_matmul_weights(segtopk_dtype dtype, const void* a_rows, int64_t a_width,
                                              int64_t a_stride, const void* b_rows, int64_t b_width,
                                              int64_t b_stride, int64_t num_rows, int32_t experts,
                                              const int64_t* offsets, segtopk_dtype out_dtype, void* out,
                                              void* stream);

/*
 * segtopk_test_expert_tile (instrumented build; host only, no CUDA call): the
 * rows of an expert that its tile `index` of segtopk_expert_matmul has, by the
 * arithmetic of the kernel: `width` of the expert's `rows` rows from `first`
 * on. An expert has ceil(rows / 256) tiles of them (for each 256 outputs).
 * Errors: SEGTOPK_ERROR_INVALID_VALUE for a number of rows or an index out of
 * range.
 */
SEGTOPK_API int segtopk_test_expert_tile(int32_t rows, int32_t index, int32_t* first, int32_t* width);

/*
 * segtopk_test_free_row (instrumented build; host only, no CUDA call): the row
 * of the result that the kernels take as number `index` of those that no
 * expert has, where the experts' rows begin at `first` and end at `end`.
 * Errors: SEGTOPK_ERROR_INVALID_VALUE.
 */
SEGTOPK_API int segtopk_test_free_row(int32_t first, int32_t end, int32_t index, int64_t* row);

/* ---------------------------------------------------------------------------
 * Layer norm, and rows in 8 bits
 * ---------------------------------------------------------------------------
 * Rows, strides, pointers and errors as for the row operators above.
 */

/* Widest row of segtopk_layer_norm. */
#define SEGTOPK_MAX_NORM_WIDTH 16384

/*
 * out[t] = (x[t] - mean[t]) * rstd[t] * weight + bias, with the mean of the
 * row's `width` values and rstd = 1 / sqrt(the mean of (x[t] - mean[t])^2 +
 * eps), both of which are written too (num_rows floats each). weight and bias
 * (NULL: none) hold `width` values of weight_dtype: dtype or F32. eps >= 0.
 */
SEGTOPK_API int segtopk_layer_norm(segtopk_dtype dtype, const void* x, int64_t num_rows, int64_t width,
                                   int64_t row_stride, segtopk_dtype weight_dtype, const void* weight,
                                   const void* bias, float eps, void* out, float* mean, float* rstd, void* stream);

/*
 * Its gradients, from that of out: of x (num_rows dense rows), of weight and
 * of bias (of weight_dtype; sums over the rows in an order that depends on the
 * sizes alone; zeros where there are no rows). mean and rstd are what the
 * forward call wrote. workspace: at least
 * segtopk_layer_norm_backward_workspace_bytes(...) bytes, 16-byte aligned
 * (host-only arithmetic; 0 for no rows and for sizes out of range).
 */
SEGTOPK_API size_t segtopk_layer_norm_backward_workspace_bytes(int64_t num_rows, int64_t width);
SEGTOPK_API int segtopk_layer_norm_backward(segtopk_dtype dtype, const void* grad_out, int64_t grad_stride,
                                            const void* x, int64_t num_rows, int64_t width, int64_t row_stride,
                                            segtopk_dtype weight_dtype, const void* weight, const float* mean,
                                            const float* rstd, void* grad_x, void* grad_weight, void* grad_bias,
                                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rows in 8 bits (e4m3) with a float scale for each block of 128 values, the
 * last block of a row in part: with a = max(the block's largest magnitude,
 * 2^-100),
 *   values[t, i] = e4m3(x[t, i] * (448 / a)),  scales[t, b] = a / 448,
 * rounded to nearest, ties to even; 448 is the largest e4m3 number. A block
 * with a NaN has a scale of NaN, one with an infinity a scale of infinity, and
 * NaN where those were. values: num_rows x width bytes; scales: num_rows x
 * ceil(width / 128). width <= 2^20, fewer than 2^31 blocks.
 */
SEGTOPK_API int segtopk_quantize_rows(segtopk_dtype dtype, const void* x, int64_t num_rows, int64_t width,
                                      int64_t row_stride, void* values, float* scales, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SEGTOPK_H_ */
