/*
 * sparsepr.h -- C ABI of the SparsePR per-call sparse-attention library (sm_100a).
 *
 * SparsePR ("Partition the Support, Reconstruct the Residual", arXiv 2608.18484)
 * replaces one softmax attention call O = softmax(s Q K^T) V by
 *   1. a response-coupled partition of keys and queries into groups
 *      (gist.science technical summary, section 2.A),
 *   2. a budgeted route of (query group, K/V group) cells and a group-contiguous
 *      permutation (same page, section 2.C; huashangw.com article, section on
 *      sparse execution),
 *   3. attention restricted to the routed cells (section 2.C),
 *   4. exact attention for 64 query-group-stratified probe rows per head, a ridge
 *      affine fit R ~ b + xB of the probe residuals inside their top singular
 *      subspace (section 2.B; huashangw.com method walkthrough), and
 *   5. the correction of every unprobed row (section 2.B).
 * The call takes Q, K, V and a target executed-pair density and returns the
 * reconstructed output (ai-feeds.com summary, 方法: 输入 / 输出).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors are device pointers unless stated.  Q, K, V and outputs named O* are
 *    bf16, contiguous [B, H, N, d] (row stride d elements), and start on a 16-byte
 *    boundary (the kernels move them with TMA; a misaligned one is SPARSEPR_EINVAL).
 *    "BH" below is B*H and every per-head array is laid out head-major ([B, H, ...]
 *    flattened).
 *  - Token indices are int32 positions in [0, N) of the original sequence.
 *  - Ownership: the caller owns every buffer.  Every entry point except
 *    sparsepr_probe_fit_noalloc allocates nothing and keeps no state between calls:
 *    their scratch memory is the caller's `workspace` (device, 256-byte aligned, at
 *    least sparsepr_workspace_bytes(p) bytes); partition, attend and probe_fit use
 *    disjoint regions of it, so attend and probe_fit may run concurrently on two
 *    streams sharing one workspace.  sparsepr_probe_fit_noalloc instead uses a fixed
 *    16 MiB device array that the library holds on every GPU that loads it (see its
 *    declaration).  sparsepr_forward (and the host entry points built on it) creates
 *    and releases a second stream and CUDA events inside the call, and
 *    sparsepr_forward_host_chunked its CUDA events (no device memory).
 *  - Asynchrony: every call only enqueues work on `stream` (a cudaStream_t; NULL
 *    is the legacy default stream) and returns.  Argument errors are detected on
 *    the host before anything is enqueued and return SPARSEPR_EINVAL or
 *    SPARSEPR_EUNSUPPORTED; a failed launch returns SPARSEPR_ECUDA.  Device-side
 *    checks (bounded waits, index checks) record an error code in the workspace;
 *    read it with sparsepr_workspace_error() after the stream has drained.  Codes:
 *    1 index out of range, 2 bounded wait ran out, 3 random-draw map overflow,
 *    4 non-finite value, 5 frame ids out of range or decreasing, 6 more than 2048
 *    k-means label corrections for one block of 16 groups in one Lloyd step (the
 *    exact re-check of near-tie rows; the call's outputs are then unspecified).
 *  - Determinism: for fixed inputs, params and seed every output is bitwise
 *    reproducible (no floating-point atomics on any output path).
 *  - Random draws (query sample, k-means seeds, probe rows) use SplitMix64
 *    (Steele, Lea & Flood 2014) with one stream per (head, purpose):
 *    state0 = mix(seed + 0xD1B54A32D192ED03 * (8*g + purpose + 1)),
 *    purpose 0 = query sample, 1 = key k-means seeds, 2 = query k-means seeds,
 *    3 = probe rows; a draw of m of n items is a partial Fisher-Yates shuffle
 *    (j = i + next() mod (n - i)).  g is the head's index in the whole layer:
 *    g = b * heads_total + head_offset + h for head h of batch element b of the
 *    call (g = b * H + h by default), so a call split by heads or batch elements
 *    (over GPUs, or in chunks) reproduces the unsplit call bit for bit.
 */
#ifndef SPARSEPR_H
#define SPARSEPR_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SPARSEPR_API __attribute__((visibility("default")))
#else
#define SPARSEPR_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SPARSEPR_OK = 0,
  SPARSEPR_EINVAL = 1,        /* invalid argument (null pointer, size out of range, density below the probe floor) */
  SPARSEPR_EUNSUPPORTED = 2,  /* valid but outside what the kernels implement (d not 64/128, too many groups, ...) */
  SPARSEPR_EWORKSPACE = 3,    /* workspace smaller than sparsepr_workspace_bytes() or misaligned */
  SPARSEPR_ECUDA = 4,         /* a CUDA runtime call or kernel launch failed */
  SPARSEPR_EDEVICE = 5        /* a device-side check failed (see sparsepr_workspace_error) */
} sparsepr_status;

/* Parameters of one attention call.  Defaults that the pages leave open are
 * readings; the recommended values per workload are listed with each field. */
typedef struct {
  int B, H, N, d;          /* batch, heads, tokens, head dim (d = 64 or 128)                        */
  int block;               /* tile rows of the permuted layout reported in block_mask (64 or 128)  */
  float density;           /* target executed-pair density rho_exec in (0, 1], probe pairs included;
                              >= 1 routes every non-empty cell                                      */
  int n_kgroups;           /* K/V groups G_k: 1..min(N,1024) is valid (else SPARSEPR_EINVAL); the
                              kernels implement G_k <= 128, more returns SPARSEPR_EUNSUPPORTED     */
  int n_qgroups;           /* query groups G_q: as G_k (valid up to min(N,1024), implemented up to
                              128)                                                                 */
  int n_samples;           /* sampled queries M_s for M_K (1..min(N,1024); default max(64, d))      */
  int n_probes;            /* probe rows per head P (1..min(N,64); the article uses 64)             */
  int eig_rank;            /* eigenpairs of M_K kept for key coordinates r_e (16 or 32; default d/4) */
  int sub_rank;            /* probe-residual subspace rank r (1..min(d, P, 64))                     */
  int kmeans_iters;        /* Lloyd assignment steps per k-means (1..64)                            */
  float ridge_lambda;      /* ridge penalty, absolute (> 0; default 1e-2)                           */
  float scale;             /* softmax scale; 0 means 1/sqrt(d)                                      */
  unsigned long long seed; /* seed of the SplitMix64 streams                                        */
  const int* frame_id;     /* NULL, or device int32 [N]: frame of each token (shared by all b, h);
                              then query q sees key k only if frame_id[k] <= frame_id[q]
                              (frame-causal, intersected with the route; the cell mass, cell cost
                              and budget count visible pairs only).  Ids must be nondecreasing in
                              token order (frame-major flattening of a video latent) and lie in
                              [0, n_frames); a violation is recorded as device error 5 and leaves
                              the outputs unspecified.  Needs N <= 65535 (32-bit cell costs).     */
  int n_frames;            /* with frame_id: number of frames, 1..64; ignored without frame_id     */
  int partition_mode;      /* 0: response-coupled partition (the method);
                              1: the semantic-grouping baseline of the pages' comparison (keys and
                              queries clustered separately on their raw vectors, same k-means
                              rules, seed streams, centroids, route and layout).  In mode 1 the
                              trace's sample_idx, metric, eigval, eigvec and key_coords are not
                              written.                                                            */
  int fit_weighted;        /* 0: uniform probe weights in the ridge fit; 1: each probe weighted by
                              n_a / (probes of its group a), normalised to mean 1 (the weighted
                              affine fit one page mentions)                                       */
  int fit_input;           /* input x of the affine map R ~ b + xB:
                              0 (default): the row's whole d-dimensional sparse output, with only
                              the correction projected onto the residual subspace (gist.science
                              2.B; huashangw.com method section: the corrected result is limited
                              to the residual directions the probes observed);
                              1: the sparse output projected on that subspace as well (x V_r)    */
  int head_offset;         /* index of this call's first head in the layer (>= 0; default 0)      */
  int heads_total;         /* heads per batch element of the layer (0: H; else >= head_offset + H);
                              with head_offset only the random streams depend on them              */
} sparsepr_params;

/* Optional debug copies of partition intermediates (any pointer may be NULL). */
typedef struct {
  int* sample_idx;          /* [BH, M_s]            sampled query rows, draw order                  */
  float* metric;            /* [BH, d, d]           M_K = Q_s^T Q_s / M_s                           */
  float* eigval;            /* [BH, r_e]            leading eigenvalues, descending                 */
  float* eigvec;            /* [BH, d, r_e]         matching eigenvectors (columns)                 */
  float* key_coords;        /* [BH, N, r_e]         y = Lambda^{1/2} U^T k                          */
  int* key_init;            /* [BH, G_k]            k-means seed rows                               */
  int* key_label_iters;     /* [T, BH, N]           key labels after every assignment step          */
  float* key_centroids;     /* [BH, G_k, d]         mean raw key per K/V group                      */
  float* query_coords;      /* [BH, N, G_k]         z = s C q                                       */
  int* query_init;          /* [BH, G_q]                                                            */
  int* query_label_iters;   /* [T, BH, N]                                                           */
  float* cell_mass;         /* [BH, G_q, G_k]       estimated retained mass per cell                */
  double* alpha;            /* [BH]                 shared mass target chosen by the route          */
} sparsepr_partition_trace;

/* Optional debug copies of probe intermediates (any pointer may be NULL). */
typedef struct {
  float* probe_o_sparse;    /* [BH, P, d]  routed-only output of the probe rows (fp32)              */
  float* probe_lse_dense;   /* [BH, P]     natural-log partition functions                          */
  float* probe_lse_sparse;  /* [BH, P]                                                              */
  float* sigma;             /* [BH, r]     singular values of the probe residual matrix             */
  float* b_sub;             /* [BH, r]     intercept in subspace coordinates                        */
} sparsepr_probe_trace;

/* Bytes of device workspace any call below needs for these params (0 if the
 * params are invalid or unsupported). */
SPARSEPR_API size_t sparsepr_workspace_bytes(const sparsepr_params* p);

/* Host-only validation of the params (no CUDA call). */
SPARSEPR_API sparsepr_status sparsepr_validate(const sparsepr_params* p);

/* Response-coupled partition, route and permutation
 * (gist.science 2.A and 2.C; huashangw.com, method and sparse-execution sections).
 *   Q, K       bf16 [B, H, N, d]
 *   perm_q/k   int32 [BH, N]     permuted position -> original token (stable by group)
 *   label_q/k  int32 [BH, N]     group of each original token
 *   qoff/koff  int32 [BH, G+1]   first permuted position of each group
 *   route      uint8 [BH, G_q, G_k]  1 = cell executed
 *   block_mask uint8 [BH, T, T]  T = ceil(N/block); tile (i, j) of the permuted layout holds a routed pair
 *   rho_exec   float [BH]        realized (routed pairs + P*N) / N^2; frame-causal: (routed visible
 *                                pairs + P*V/N) / V with V the visible pairs of the causal mask
 *   trace      optional, may be NULL                                                   */
SPARSEPR_API sparsepr_status sparsepr_partition(const sparsepr_params* p, const void* Q, const void* K,
                                   int* perm_q, int* perm_k, int* label_q, int* label_k,
                                   int* qoff, int* koff, unsigned char* route,
                                   unsigned char* block_mask, float* rho_exec,
                                   const sparsepr_partition_trace* trace,
                                   void* workspace, size_t ws_bytes, void* stream);

/* Attention restricted to the routed cells (gist.science 2.C):
 *   O_sparse(q) = sum over keys k with route[label_q(q), label_k(k)] of softmax(s q.k) v_k,
 * written in ORIGINAL token order (bf16 [B, H, N, d]); lse = ln sum exp(s q.k) over the
 * same keys (float [BH, N]).  Inputs are the partition outputs above.                 */
SPARSEPR_API sparsepr_status sparsepr_attend(const sparsepr_params* p, const void* Q, const void* K,
                                const void* V, const int* perm_q, const int* perm_k,
                                const int* qoff, const int* koff, const unsigned char* route,
                                void* O_sparse, float* lse,
                                void* workspace, size_t ws_bytes, void* stream);

/* Exact probes and the residual fit (gist.science 2.B; huashangw.com method section).
 *   probe_idx      int32 [BH, P]    probe rows (original indices), group order then draw order
 *   probe_o_dense  float [BH, P, d] exact dense output of the probe rows
 *   b_full         float [BH, d]    b V_r^T (intercept in output space)
 *   Vr             float [BH, d, r] orthonormal basis of the residual subspace (zero columns
 *                                   where the singular value is <= 1e-6 of the largest)
 *   W              float [BH, d, r] ridge slope, residual coordinates = x W
 *   Bmat           float [BH, d, d] optional (may be NULL): the pages' B = W V_r^T
 * Depends only on the partition (not on sparsepr_attend's output).                     */
SPARSEPR_API sparsepr_status sparsepr_probe_fit(const sparsepr_params* p, const void* Q, const void* K,
                                   const void* V, const int* label_k, const int* perm_q,
                                   const int* qoff, const unsigned char* route,
                                   int* probe_idx, float* probe_o_dense, float* b_full,
                                   float* Vr, float* W, float* Bmat,
                                   const sparsepr_probe_trace* trace,
                                   void* workspace, size_t ws_bytes, void* stream);

/* sparsepr_probe_fit without a workspace: allocates nothing and uses no caller scratch.
 * The paper has no counterpart; this variant exists for callers that cannot call
 * cudaMalloc (runtimes that fix their device memory plan at start-up and forbid later
 * allocation, or host code where an allocation, which can synchronize the device, is not
 * allowed).  Arguments and outputs are those of sparsepr_probe_fit minus the trace and the
 * workspace; results agree with it up to floating-point summation order.
 * Frame-causal params (frame_id != NULL) are refused with SPARSEPR_EUNSUPPORTED, and Q, K,
 * V must be 16-byte aligned (else SPARSEPR_EINVAL), both before any work is enqueued.
 * Scratch: a 16 MiB device array owned by the library, present on every GPU that loads
 * it until the process exits.  With S key splits it holds
 *   B*H*(n_probes*(4*d + 12) + S*64*(8*d + 16)) bytes (each region rounded up to 256)
 * plus a 256-byte error word; S starts at the workspace entry point's split count for N
 * and shrinks until the problem fits, and a problem that does not fit even with S = 1
 * returns SPARSEPR_EUNSUPPORTED before any work is enqueued.  The first call on a device
 * looks up the array's device address (cudaGetSymbolAddress, with that device current)
 * and keeps it for the life of the process (a cudaDeviceReset invalidates it); make that
 * first call before any stream capture.  All calls share the one array and it keeps the
 * previous call's contents: the call clears its error word and rewrites every other byte
 * before reading it; calls that overlap on the GPU, on other streams or from other host
 * threads, race and must be serialized by the caller.  A device-side failure (a bounded
 * wait that ran out, an index out of range, a failed random draw) sets b_full, Vr, W and
 * Bmat of every head to NaN instead of leaving stale values.                           */
SPARSEPR_API sparsepr_status sparsepr_probe_fit_noalloc(const sparsepr_params* p, const void* Q,
                                                        const void* K, const void* V,
                                                        const int* label_k, const int* perm_q,
                                                        const int* qoff, const unsigned char* route,
                                                        int* probe_idx, float* probe_o_dense,
                                                        float* b_full, float* Vr, float* W,
                                                        float* Bmat, void* stream);

/* Correction of every unprobed row and restoration of the probe rows (gist.science 2.B):
 *   O(q) = x + b_full + (x W) V_r^T   with x = O_sparse(q), for q not a probe;
 *   O(q) = probe_o_dense              for probe rows.
 * O is bf16 [B, H, N, d] and may alias O_sparse.                                       */
SPARSEPR_API sparsepr_status sparsepr_reconstruct(const sparsepr_params* p, const void* O_sparse,
                                     const int* probe_idx, const float* probe_o_dense,
                                     const float* b_full, const float* Vr, const float* W,
                                     void* O, void* stream);

/* The whole call (partition -> attend -> probe_fit -> reconstruct) on device buffers,
 * with every intermediate kept in the workspace (sparsepr_forward_workspace_bytes).
 * rho_exec (float [BH]) may be NULL.  The probe path (sparsepr_probe_fit's kernels) runs
 * on a second stream that the call creates, forks from `stream` after the partition and
 * joins back before the correction, so it overlaps the routed attention; the stream and
 * its events are released before the call returns (freed once their work completes).
 * If they cannot be created, or `stream` is being captured into a CUDA graph, everything
 * runs on `stream`.  The results do not depend on the overlap.                         */
SPARSEPR_API size_t sparsepr_forward_workspace_bytes(const sparsepr_params* p);
SPARSEPR_API sparsepr_status sparsepr_forward(const sparsepr_params* p, const void* Q, const void* K,
                                 const void* V, void* O, float* rho_exec,
                                 void* workspace, size_t ws_bytes, void* stream);

/* sparsepr_forward from HOST buffers: copies Q, K, V (host, bf16 [B,H,N,d]; pinned memory
 * for asynchronous copies) into the caller's device staging buffer qkv_dev (3 tensors,
 * 3*BH*N*d bf16), runs the call into o_dev (device, bf16), and copies the result to
 * O_host.  Everything is enqueued on `stream`; the caller synchronizes.               */
SPARSEPR_API sparsepr_status sparsepr_forward_host(const sparsepr_params* p, const void* Q_host,
                                      const void* K_host, const void* V_host, void* O_host,
                                      void* qkv_dev, void* o_dev,
                                      void* workspace, size_t ws_bytes, void* stream);

/* sparsepr_forward_host as a pipeline over head chunks, so that the host<->device copies
 * of one chunk run beside the compute of another.  The B*H heads (flattened b*H + h) are
 * split into n_chunks (1..min(B*H, 512)) consecutive ranges of ceil(B*H / n_chunks) heads
 * (with head_offset / heads_total set, also at every batch element).  Chunk c's three
 * host-to-device copies (one cudaMemcpyAsync per tensor) go on copy_in_stream, its call
 * (sparsepr_forward with B = 1 over the chunk's heads, head_offset = their layer index, so
 * every output equals the unsplit call's bit for bit) on `stream`, and the copy of its O
 * back to O_host on copy_out_stream.  The copies in start after the work already enqueued
 * on `stream`; `stream` completes after the last copy out, so synchronizing `stream` is
 * enough.  A NULL copy stream means `stream` (no overlap).
 *   qkv_dev   device bf16 [3][B, H, N, d] staging of Q, K, V; o_dev device bf16 [B, H, N, d]
 *   workspace sparsepr_forward_workspace_bytes of the params of one chunk (B = 1,
 *             H = ceil(B*H / n_chunks)), shared by the chunks (their compute is serialized
 *             on `stream`); its error word is cleared once and collects every chunk's
 *             device errors
 * Host buffers should be pinned for the copies to be asynchronous.  The call creates its
 * CUDA events and releases them before returning (they are freed once they complete).  */
SPARSEPR_API sparsepr_status sparsepr_forward_host_chunked(const sparsepr_params* p, const void* Q_host,
                                                           const void* K_host, const void* V_host,
                                                           void* O_host, void* qkv_dev, void* o_dev,
                                                           int n_chunks, void* workspace, size_t ws_bytes,
                                                           void* stream, void* copy_in_stream,
                                                           void* copy_out_stream);

/* Dense softmax attention on the same machinery (the comparator for the sparse call):
 * O = softmax(s Q K^T) V (bf16 [B,H,N,d]), lse float [BH, N] (may be NULL); with frame ids,
 * each query attends to the keys of its own and earlier frames.  Uses only the first bytes
 * of the workspace: the error word (256 bytes; the workspace may then be NULL) and, with
 * frame ids, the frame ends (512 bytes in all, required).                              */
SPARSEPR_API sparsepr_status sparsepr_dense_attention(const sparsepr_params* p, const void* Q,
                                         const void* K, const void* V, void* O, float* lse,
                                         void* workspace, size_t ws_bytes, void* stream);

/* Device-side error code recorded in the workspace (0 = none) and its reset.  The code
 * is sticky until cleared; sparsepr_partition and sparsepr_forward clear it when they
 * start.  Both functions synchronize `stream`.                                         */
SPARSEPR_API int sparsepr_workspace_error(const sparsepr_params* p, void* workspace, void* stream);
SPARSEPR_API sparsepr_status sparsepr_workspace_clear_error(const sparsepr_params* p, void* workspace,
                                               void* stream);

/* ===========================================================================
 * Rollouts frame by frame: rotary positions and a paged K/V cache
 * ===========================================================================
 * A rollout that generates its frames (or tokens) one after another keeps the keys and
 * values of what it has generated in pages instead of calling sparsepr_forward on the
 * whole sequence again: each step rotates its new queries and keys (sparsepr_rope, or
 * inside sparsepr_cache_append), appends the keys and values to the pages, and attends
 * from the new tokens to the cache (sparsepr_paged_attention), either to all of it or to
 * the pages that a cheap score selects (sparsepr_page_select).
 *
 * The conventions at the top of this file hold (ownership, streams, argument errors,
 * determinism), with these differences: tensors are bf16 or fp16 (rotary positions: fp32
 * too), their rows are packed tokens with strides in the params, and the workspace is
 * sparsepr_paged_workspace_bytes() with its own error query, sparsepr_paged_error().
 * The entry points of this section never clear the error word except for
 * sparsepr_paged_clear_error(): clear it once after allocating the workspace.  Calls that
 * may overlap on the GPU need a workspace each.  All calls can be captured into CUDA graphs;
 * a graph's calls keep the workspace they were captured with.                                        */

/* element types */
#define SPARSEPR_BF16 0
#define SPARSEPR_FP16 1
#define SPARSEPR_FP32 2

/* Rotary positions.  Pair i (0 <= i < rot_dim/2) of a row of token n turns by the angle
 *   t = 2 pi * pos[axis(i)][n] * freq[i]                     (freq in turns per position)
 *   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_a sin t + x_b cos t)
 * with (a, b) = (i, i + rot_dim/2) (layout 0, halves) or (2i, 2i + 1) (layout 1,
 * interleaved); elements rot_dim .. d-1 are copied.  The pairs are divided into n_axes
 * consecutive sections of axis_dim[a]/2 pairs (time, height, width of a video latent; one
 * axis for text-like sequences).  Angles are formed and reduced in 64 bits and are off by a
 * few 2^-53 |pos| rad: below fp32's half step of 2^-24 up to positions of 2^27, 10^-6 at 2^31
 * (16-bit rows round more coarsely than that at every position).                       */
typedef struct {
  int B, H, N, d;          /* batch, heads, tokens (0 is allowed), head dim (2..512)                */
  int H2;                  /* heads of the second tensor of the call (0: none)                      */
  int dtype;               /* SPARSEPR_BF16, SPARSEPR_FP16 or SPARSEPR_FP32                         */
  int rot_dim;             /* rotated elements of each row: even, 2..d                              */
  int layout;              /* 0: halves, 1: interleaved                                             */
  int n_axes;              /* position axes, 1..3                                                   */
  int axis_dim[3];         /* rotated elements per axis: even, >= 2, summing to rot_dim             */
  int pos_batched;         /* 0: pos is int32 [n_axes, N], 1: int32 [n_axes, B, N]                  */
  int scaling;             /* of the frequencies theta^(-2j/axis_dim), j the pair within its axis:
                              0 none; 1 linear: divided by factor;
                              2 base: theta replaced by theta factor^(axis_dim/(axis_dim - 2));
                              3 by parts: pairs that turn beta_fast times or more within orig_len
                              positions keep their frequency, those that turn beta_slow times or
                              less have it divided by factor, and those in between mix the two: with
                              c(t) = axis_dim ln(orig_len/(2 pi t)) / (2 ln theta) the pair that turns
                              t times, lo = max(floor c(beta_fast), 0), hi = min(ceil c(beta_slow),
                              axis_dim - 1), the frequency times 1 - r + r/factor with
                              r = (j - lo) / max(hi - lo, 0.001) limited to [0, 1]                 */
  int orig_len;            /* scaling 3: positions the frequencies were made for (>= 1)             */
  double theta;            /* > 0 (10000)                                                           */
  double factor;           /* > 0 (1)                                                               */
  double beta_fast, beta_slow; /* scaling 3: beta_fast > beta_slow > 0 (32 and 1)                   */
  double magnitude;        /* m; 0 means 1, or 0.1 ln(factor) + 1 with scaling 3 and factor > 1     */
  long long x_stride[3], y_stride[3];    /* element strides of batch, head and token of the first
                              tensor's input and output; all three 0 means contiguous [B,H,N,d].
                              The last dimension is contiguous; an output stride may not be 0.     */
  long long x2_stride[3], y2_stride[3];  /* the same for the second tensor                          */
} sparsepr_rope_params;

/* Fills freq[rot_dim/2] (HOST memory, turns per position) from the params; copy it to the
 * device once and pass it to the calls below.  No CUDA call.                           */
SPARSEPR_API sparsepr_status sparsepr_rope_frequencies(const sparsepr_rope_params* p, double* freq_host);

/* Host-only validation of the params (no CUDA call). */
SPARSEPR_API sparsepr_status sparsepr_rope_validate(const sparsepr_rope_params* p);

/* y = rotation of x (and y2 of x2, with H2 heads, when H2 > 0), one launch for both.
 * pos and freq (double [rot_dim/2]) are device pointers.  y may be x (in place) if their
 * strides are equal; any other overlap is the caller's error.  No workspace.           */
SPARSEPR_API sparsepr_status sparsepr_rope(const sparsepr_rope_params* p, const void* x, const int* pos,
                                           const double* freq, void* y, const void* x2, void* y2, void* stream);

/* Gradient of sparsepr_rope: dx = m R(-t) dy (x_stride describes dy, y_stride dx). */
SPARSEPR_API sparsepr_status sparsepr_rope_backward(const sparsepr_rope_params* p, const void* dy, const int* pos,
                                                    const double* freq, void* dx, const void* dy2, void* dx2,
                                                    void* stream);

/* A step of a rollout over B sequences with a paged K/V cache.
 *   k_pages, v_pages  [n_pages, Hkv, page, d]  contiguous, 16-byte aligned
 *   k_mean            [n_pages, Hkv, d]        mean key of each page's rows in use
 *   page_table        int32 [B, max_pages]     page holding rows page*j .. page*j+page-1 of
 *                                              sequence b (entries past its length are not read)
 *   q_start           int32 [B+1]              first new token of each sequence among the T packed
 *                                              rows (q_start[0] >= 0, nondecreasing, <= T; rows that
 *                                              belong to no sequence are neither read nor written)
 *   kv_len            int32 [B]                cached rows of each sequence, its new tokens included
 * New token i of sequence b (n_b of them) has position kv_len[b] - n_b + i and row
 * q_start[b] + i.  A negative position (n_b > kv_len[b]) is a token without a slot: it is not
 * appended and, unless frame = 0, sees no key.                                          */
typedef struct {
  int B;                   /* sequences, 1..65536                                                   */
  int Hq, Hkv;             /* query heads and key/value heads; Hkv divides Hq, query head h reads
                              key/value head h / (Hq/Hkv)                                           */
  int d;                   /* head dim, 64 or 128                                                   */
  int dtype;               /* SPARSEPR_BF16 or SPARSEPR_FP16                                        */
  int page;                /* rows per page: 16, 32, 64 or 128                                      */
  int n_pages;             /* pages in the pool                                                     */
  int max_pages;           /* row length of page_table (max_pages * page <= 2^30)                   */
  int T;                   /* packed rows of new tokens (0 is allowed)                              */
  int max_chunk;           /* no sequence of the call has more new tokens than this (>= 1); it picks
                              the kernel, and a longer sequence is device error 1                   */
  int frame;               /* mask: a token at position x sees the keys at positions y with
                              floor(y/frame) <= floor(x/frame): 1 token-causal, the tokens of a frame
                              for a frame-causal rollout; 0: every cached key                       */
  float scale;             /* softmax scale; 0 means 1/sqrt(d)                                      */
  int q_block;             /* selection: consecutive new tokens of a sequence that share a list    */
  int n_select;            /* selection: pages of a list (0: no selection)                          */
  int n_sink, n_recent;    /* selection: leading and trailing visible pages that every list holds
                              (n_sink + n_recent <= n_select)                                       */
  long long q_stride[2], o_stride[2]; /* element strides of token and head of Q and O; both 0 means
                              contiguous [T, Hq, d].  Multiples of 8.                               */
  long long k_stride[2], v_stride[2]; /* the same for the new K and V ([T, Hkv, d])                 */
} sparsepr_cache_params;

/* Host-only validation (no CUDA call), and the workspace of the calls below (0 if invalid). */
SPARSEPR_API sparsepr_status sparsepr_cache_validate(const sparsepr_cache_params* p);
SPARSEPR_API size_t sparsepr_paged_workspace_bytes(const sparsepr_cache_params* p);

/* Writes the new K and V rows into their page slots and the mean key of every touched page
 * (over its rows in use, taken of the stored keys in a fixed order, so that it does not
 * depend on how the rows were split into calls).  With rope (NULL: none) the keys are
 * rotated on the way: rope's rot_dim, layout, axes and magnitude count, pos is int32
 * [n_axes, T] and rope_freq double [rot_dim/2] (both device); its other fields are not read
 * except that d must agree.  Pages being written must belong to one sequence of the call.
 * A page id out of [0, n_pages) is device error 1 and its rows are not written; a kv_len out
 * of [0, max_pages * page], more than max_chunk new tokens or rows out of [0, T) are device
 * error 1 and nothing of that sequence is written.                                      */
SPARSEPR_API sparsepr_status sparsepr_cache_append(const sparsepr_cache_params* p, const void* K, const void* V,
                                                   const int* q_start, const int* kv_len, const int* page_table,
                                                   void* k_pages, void* v_pages, void* k_mean,
                                                   const sparsepr_rope_params* rope, const int* pos,
                                                   const double* rope_freq, void* workspace, size_t ws_bytes,
                                                   void* stream);

/* Lists of pages for sparsepr_paged_attention.  A unit is q_block consecutive new tokens of
 * one sequence (the last one may be shorter); units are numbered sequence by sequence, and
 * there are at most sparsepr_select_units(p) = (T + (q_block - 1) B) / q_block of them (min T).
 * For a unit
 * and key/value head the score of a page is (mean of the unit's query rows over its tokens
 * and the query heads of that key/value head) . k_mean[page], summed in 64 bits.  The pages
 * that hold a key visible to the unit's last token take part; the first n_sink and the last
 * n_recent of them are kept, and the best scores fill the list up to n_select (ties to the
 * lowest page; a page whose mean, or a unit whose mean query, has an element that is not finite
 * has no score and counts as the lowest).
 *   sel       int32 [units, Hkv, n_select]  page indices within the sequence, ascending, -1 behind
 *   sel_count int32 [units, Hkv]            entries of each list
 * Rows of units that do not exist are left as they were.  A page id out of [0, n_pages) is
 * device error 1 and counts as the lowest score.  With more than 8,192 pages per sequence the
 * lists are made in batches, so that the workspace holds at most 256 MB of scores and 256 MB
 * of keys (or 12 bytes per page of one list, if that is more).                          */
SPARSEPR_API int sparsepr_select_units(const sparsepr_cache_params* p);
SPARSEPR_API sparsepr_status sparsepr_page_select(const sparsepr_cache_params* p, const void* Q, const int* q_start,
                                                  const int* kv_len, const int* page_table, const void* k_mean,
                                                  int* sel, int* sel_count, void* workspace, size_t ws_bytes,
                                                  void* stream);

/* Attention of the new tokens over the cache:
 *   O(i, h) = sum over visible keys j of softmax_j(s q.k_j) v_j,  lse(i, h) = ln sum exp(s q.k_j)
 * (O [T, Hq, d]; lse float [T, Hq], may be NULL), over the pages of the token's list when sel
 * and sel_count are given (n_select > 0), else over the whole cache.  O must not overlap Q.  A
 * token that sees no key gets O = 0 and lse = -inf.  Keys past kv_len, and keys that no token of a block of
 * rows sees, are never used, whatever their slots hold (a NaN or an infinity in a value row
 * that some tokens of a block see can reach the block's other rows).
 * A page id out of [0, n_pages), a list that is not strictly ascending or leaves the visible
 * pages, a kv_len out of [0, max_pages * page] or a sequence of more than max_chunk new tokens
 * is device error 1; the rows that depend on it become NaN (of such a sequence, those that are
 * written).                                                                        */
SPARSEPR_API sparsepr_status sparsepr_paged_attention(const sparsepr_cache_params* p, const void* Q,
                                                      const int* q_start, const int* kv_len,
                                                      const int* page_table, const void* k_pages,
                                                      const void* v_pages, const int* sel, const int* sel_count,
                                                      void* O, float* lse, void* workspace, size_t ws_bytes,
                                                      void* stream);

/* Error word of a paged workspace (0 = none; codes as above; -1 if it cannot be read) and
 * its reset.  The query synchronizes `stream`; the reset only enqueues.                 */
SPARSEPR_API int sparsepr_paged_error(const void* workspace, void* stream);
SPARSEPR_API sparsepr_status sparsepr_paged_clear_error(void* workspace, void* stream);

/* Human-readable status; sparsepr_last_error() gives the detail of the most recent
 * failing call on this host thread (static storage, never NULL).                      */
SPARSEPR_API const char* sparsepr_status_string(sparsepr_status s);
SPARSEPR_API const char* sparsepr_last_error(void);

/* Number of kernel launches the last successful call on this host thread enqueued. */
SPARSEPR_API int sparsepr_last_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* SPARSEPR_H */
