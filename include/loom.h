/*
 * loom.h -- C ABI of the MI355X (gfx950, CDNA4) streaming-reduction library.
 *
 * The library computes the data-parallel hot path described by the Loom pages
 * "Tune loop unrolling and pipelining" (TUNE), "Functions and structured
 * control flow" (CTRL) and "Kernels and launch configuration" (LAUNCH): a
 * streaming reduction over records in memory -- row-tiled f32 sums with a
 * subgroup (wave64) reduction per row, full 8-row tiles with a separate ragged
 * tail, read-ahead of the next records -- and its extension to packed
 * signed-byte (int8) dequantization with dot accumulation.
 *
 * Conventions for every entry point
 * ---------------------------------
 *  - Return LOOM_OK (0) or a negative loom_status.  All argument checks run on
 *    the host before anything is enqueued; on error nothing is launched and no
 *    output is touched.  Sizes and counts are checked first (LOOM_ERR_RANGE,
 *    LOOM_ERR_SHAPE), including the launch grid's limit of fewer than 2^32
 *    work-items (see each call); a call with nothing to do (no rows,
 *    elements, segments, outputs or tokens) then returns LOOM_OK without
 *    looking at its pointers;
 *    otherwise required pointers (LOOM_ERR_NULL) and then alignment
 *    (LOOM_ERR_ALIGN) are checked.
 *  - Data pointers are device pointers (HIP allocations of the current device,
 *    e.g. a torch tensor's data_ptr()).  The caller owns all memory.  The
 *    library keeps no pointer after returning and allocates no device memory,
 *    except loom_segment_sums in its split and longest-first launches, whose
 *    workspace comes from HIP's stream-ordered allocator (see there;
 *    loom_segment_sums_noalloc never allocates).
 *  - `stream` is a hipStream_t (NULL = the null stream).  Work is enqueued
 *    asynchronously on it; outputs are ready once the stream has reached the
 *    enqueued work.  A device-side fault is reported by later HIP calls, not
 *    by the return code; LOOM_ERR_DEVICE means the launch itself was refused
 *    (the thread's last HIP error is cleared before each launch, so an error
 *    left by an earlier, unrelated HIP call is never reported as this one).
 *  - Calls are thread-safe: the shared state is an immutable table and, for
 *    loom_segment_sums_noalloc, a lock-guarded per-device address cache and
 *    the static device array (calls of it that overlap on one GPU race; see
 *    there).
 *  - Matrices are row-major.  Packed int8: an int32 word j of a row holds the
 *    elements 4j..4j+3, element 4j+b in byte b (little-endian), two's
 *    complement -- exactly the bytes of an int8 array viewed as int32.
 */
#ifndef LOOM_H
#define LOOM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum loom_status {
    LOOM_OK = 0,
    LOOM_ERR_NULL = -1,           /* a required pointer is NULL                          */
    LOOM_ERR_RANGE = -2,          /* a size or count outside its documented range        */
    LOOM_ERR_ALIGN = -3,          /* a pointer or stride not aligned as documented       */
    LOOM_ERR_SHAPE = -4,          /* inconsistent shape (e.g. k not a multiple of 4)     */
    LOOM_ERR_UNKNOWN_EXPORT = -5, /* no kernel exports this name                         */
    LOOM_ERR_TOKEN = -6,          /* invalid launch-config token or workload arity       */
    LOOM_ERR_DEVICE = -7          /* the HIP runtime refused the launch                  */
} loom_status;

/* Static, human-readable text for a status code (never NULL). */
const char *loom_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int loom_version(void);

/* ------------------------------------------------------------------------ *
 * Launch configuration (LAUNCH §A kernel owns two signatures, §Workload is  *
 * not workgroup count, §Evaluate the compiled launch contract).             *
 *                                                                           *
 * Each kernel owns the mapping from its logical workload (element, row or   *
 * segment counts) to a physical grid.  An embedding resolves an export name  *
 * to a token once, then evaluates the geometry for any workload without     *
 * compiling anything.  The entry points below use the same evaluation, so   *
 * the host never duplicates the grid arithmetic.                            *
 * ------------------------------------------------------------------------ */
typedef struct loom_launch_config {
    uint32_t workgroups[3];          /* grid, in workgroups                       */
    uint32_t workgroup_size[3];      /* work-items per workgroup                  */
    uint32_t cluster_size[3];        /* always {1,1,1}: gfx950 has no clusters    */
    uint32_t subgroup_size;          /* 64: gfx950 waves are 64 wide              */
    uint32_t workgroup_storage_bytes;/* LDS the kernel needs per workgroup        */
} loom_launch_config;

/* Export names and their workload signatures (each an int64 passed as its
 * uint64 bit pattern):
 *   "copy_f32"        (n)
 *   "row_sum_tiles"   (count)
 *   "row_sums"        (rows, cols)
 *   "segment_sums"    (segments, cols, total_rows)
 *   "i8_dequant_dot"  (rows, k, batch)
 *   "packed_dot"      (outputs, count, streams)
 *   "sum_guarded_rows" (count)
 *   "routed_combine"  (tokens, routes, hidden)
 *   "quantize_rows"   (rows, cols)
 *   "i8_matmul", "i8_gated_projection" (rows, k, tokens)
 *   "i8_gated_projection_backward" (rows, k, tokens): its first kernel
 *   "route_experts" (tokens, experts, groups, top_k)
 *   "route_experts_backward" (tokens, experts, 1, top_k)
 *   "group_routes"    (pairs, experts), pairs = tokens * routes
 *   "i4_matmul"       (rows, k, tokens, group)
 *   "i4_expert_matmul", "i4_expert_gated_projection"
 *                     (rows, k, pairs, group, experts)
 * lookup: LOOM_ERR_NULL if a pointer is NULL, LOOM_ERR_UNKNOWN_EXPORT if no
 * kernel has that name.  The token stays valid for the life of the process. */
int loom_launch_config_lookup(const char *export_name, uint32_t *token);

/* Evaluates the launch configuration of `token` for the given workload.
 * Pure host arithmetic; no device call.  LOOM_ERR_TOKEN for an unknown token
 * or a workload_count that differs from the export's arity, LOOM_ERR_RANGE
 * for a negative workload value or a grid beyond the hardware limits.
 * A workload with nothing to do yields workgroups {0,1,1}. */
int loom_launch_config_invoke(uint32_t token, const uint64_t *workload_bits,
                              size_t workload_count, loom_launch_config *out);

/* ------------------------------------------------------------------------ *
 * Guarded over-dispatched copy (LAUNCH §Over-dispatch safely and preserve   *
 * the proof).  out[i] = in[i] for 0 <= i < n, on ceil(n/256) workgroups of   *
 * 256 work-items; work-items at or beyond n touch nothing, so out[n..] is   *
 * left as it was (1009 elements run on 4 workgroups).                       *
 *   in, out : f32[n], device, 4-byte aligned; may be NULL only when n == 0  *
 *   n       : 0 <= n <= 2^32 - 256, so the grid stays below 2^32           *
 *             work-items (LOOM_ERR_RANGE otherwise)                         *
 * ------------------------------------------------------------------------ */
int loom_copy_f32(const float *in, float *out, int64_t n, void *stream);

/* ------------------------------------------------------------------------ *
 * Tiled row sum of one 32-lane tile (TUNE §Derive full tiles from a ragged  *
 * loop, @guide.sum_full_tiles).  For lane l < 32:                           *
 *     sums[l] = initial[l] + sum over rows r < final_row of rowsum(r)       *
 * where rowsum(r) is the subgroup reduction of values[r][0..31], rows are   *
 * taken in full tiles of 8 in row order, final_row = 8*floor(count/8) and   *
 * tail_count = count mod 8.  The tail rows [final_row, count) are NOT       *
 * summed and NOT read: they are returned for a separate cleanup.            *
 *   values     : f32[rows_alloc][32], device, 4-byte aligned                *
 *   rows_alloc : rows allocated, 0 <= rows_alloc <= 2^26                    *
 *   count      : logical row count, 0 <= count <= rows_alloc (the page's    *
 *                inclusive range assumption, checked: LOOM_ERR_RANGE)       *
 *   initial    : f32[32] per-lane start value, or NULL for 0.0              *
 *   sums       : f32[32] output                                             *
 *   final_row, tail_count : int32[1] outputs, device                        *
 * ------------------------------------------------------------------------ */
int loom_row_sum_tiles(const float *values, int64_t rows_alloc, int64_t count,
                       const float *initial, float *sums, int32_t *final_row,
                       int32_t *tail_count, void *stream);

/* ------------------------------------------------------------------------ *
 * Streaming row sums (TUNE §Derive full tiles, §Give each motif its own     *
 * schedule, §Read-ahead; CTRL §Pipeline reads ahead of ordered computation) *
 *     out[r] = sum_{c < cols} x[r*row_stride + c],   0 <= r < rows          *
 * Every row is streamed with coalesced loads read ahead of the              *
 * accumulation and finished by cross-lane reductions; how rows map to the   *
 * GPU depends on their width: 1-128 floats are packed several to a 64-lane  *
 * record; 129-768 floats run in full 8-row tiles plus one guarded tail      *
 * tile; a row of 769 floats or more gets a workgroup of its own whose wave  *
 * totals are added in wave order.  f32 accumulation; the summation          *
 * order inside a row is a fixed tree, the same on every call (error         *
 * <= 1e-5 * sum|x| for the documented sizes).                               *
 *   x          : f32, device, 4-byte aligned (16-byte alignment of x and    *
 *                row_stride % 4 == 0 select 128-bit loads)                  *
 *   rows, cols : 0 <= rows < 2^31, 0 <= cols < 2^31; LOOM_ERR_RANGE also    *
 *                when the grid would reach 2^32 work-items, as              *
 *                loom_launch_config_invoke reports for (rows, cols): only   *
 *                past 2^30 - 16 rows of at most 768 floats                  *
 *   row_stride : elements between row starts, row_stride >= cols            *
 *                (LOOM_ERR_SHAPE); 4 * rows * row_stride must fit in an     *
 *                int64 (LOOM_ERR_RANGE)                                     *
 *   out        : f32[rows], device                                          *
 * ------------------------------------------------------------------------ */
int loom_row_sums(const float *x, int64_t rows, int64_t cols, int64_t row_stride,
                  float *out, void *stream);

/* ------------------------------------------------------------------------ *
 * Per-segment column sums (TUNE §Keep one checked source for experiments:   *
 * each lane sums its column over the rows, in row order; §Derive full       *
 * tiles: full 8-row tiles then the tail).                                   *
 *     out[s][c] = sum_{offsets[s] <= r < offsets[s+1]} x[r][c]              *
 *     tail_counts[s] = (offsets[s+1] - offsets[s]) mod 8                    *
 * Each column accumulates its rows in row order in f32, so every output is  *
 * the in-order recurrence bit for bit (an empty segment gives +0.0) --      *
 * except for a few long segments: when segments x ceil(cols / 256) < 192    *
 * and the segments average at least 1024 rows (total_rows / segments), each *
 * segment is split into P contiguous parts of at least 512 rows on average  *
 * (P * segments * ceil(cols / 256) <= 4096), each part summed in row order, *
 * and the part sums added in a fixed order.  With cols <= 512 and P >= 16,  *
 * P is a multiple of 8 and the sums of each run of 8 consecutive parts are  *
 * added in part order, leaving n = P / 8 partials per segment; otherwise    *
 * the n = P part sums are the partials.  The n partials are added as        *
 * contiguous groups of ceil(n / 16) in order, then the group sums in group  *
 * order: the same bits on every call, within 1e-5 * sum|x| of the in-order  *
 * sum.  The partials (4 * segments * n * cols bytes, at most 4 MiB) are     *
 * taken from HIP's stream-ordered allocator on `stream` (hipMallocAsync /   *
 * hipFreeAsync).  A launch that is not split, of 2 to 2^15 segments         *
 * averaging at least 512 rows and of at least 2^26 floats, first sorts the  *
 * segments by length (a one-workgroup pass) so its waves take them longest  *
 * first; the order index (4 * segments bytes) is taken the same way.  These *
 * are the only cases where a call allocates device memory; neither changes  *
 * a bit of output.                                                          *
 *   x           : f32[total_rows][cols], device, row-major, 4-byte aligned  *
 *   total_rows  : rows in x, 0 <= total_rows <= 2^40                        *
 *   offsets     : int64[segments+1], device, CSR row offsets.  A segment    *
 *                 with offsets[s] > offsets[s+1], offsets[s] < 0 or         *
 *                 offsets[s+1] > total_rows reads nothing; its outputs are  *
 *                 set to NaN and its tail count to -1.                      *
 *   segments    : 0 <= segments < 2^31 - 1                                  *
 *   cols        : 0 <= cols <= 2^20                                         *
 *   out         : f32[segments][cols], device                               *
 *   tail_counts : int32[segments], device, or NULL                          *
 * LOOM_ERR_DEVICE also when the stream-ordered allocation fails.            *
 * ------------------------------------------------------------------------ */
int loom_segment_sums(const float *x, int64_t total_rows, const int64_t *offsets,
                      int64_t segments, int64_t cols, float *out,
                      int32_t *tail_counts, void *stream);

/* ------------------------------------------------------------------------ *
 * For callers that cannot allocate device memory -- code under HIP graph    *
 * capture, tight serving loops, harnesses that forbid hipMalloc: the same   *
 * operation, arguments, checks and results (the same bits) as              *
 * loom_segment_sums, but a split launch's partials and a longest-first     *
 * launch's order index live in the library's own static device array of    *
 * 4 MiB (one per GPU the library runs on, kept until the process ends)      *
 * instead of stream-ordered memory, so no call allocates.  Every call on a  *
 * GPU shares that GPU's array and it keeps the last call's contents (each   *
 * launch writes every word of it that it reads):                            *
 * calls that may overlap on one GPU -- on different streams or threads --   *
 * race and must be ordered by the caller.  LOOM_ERR_RANGE if a split would  *
 * need more than the array holds (the split rule keeps every launch within  *
 * it).                                                                      *
 * ------------------------------------------------------------------------ */
int loom_segment_sums_noalloc(const float *x, int64_t total_rows, const int64_t *offsets,
                              int64_t segments, int64_t cols, float *out,
                              int32_t *tail_counts, void *stream);

/* ------------------------------------------------------------------------ *
 * Packed signed-byte dequantization with dot accumulation (TUNE §Apply the  *
 * same controls to a packed dot product; scales factored out of the sum).   *
 *     acc[r][b] = sum_{i < k} w[r][i] * x[b][i]          (exact, int32)     *
 *     out[r][b] = (f32(acc[r][b]) * w_scale[r]) * x_scale[b]                *
 * with each product rounded once to f32; when x_scale is NULL the second    *
 * product is skipped.  One vector runs a v_dot4 (int8x4) GEMV: rows of up  *
 * to 512 bytes packed several to a 1 KiB record, most rows of 3 to 12 KiB   *
 * a workgroup per row, other rows a wave per block of rows.  Several        *
 * vectors run an int8 MFMA kernel.  The results are the same bits either    *
 * way.                                                                      *
 *   w       : int32[rows][k/4] packed int8 weights, device, 4-byte aligned  *
 *   w_scale : f32[rows], device                                             *
 *   x       : int32[batch][k/4] packed int8 activations, device             *
 *   x_scale : f32[batch], device, or NULL (= 1)                             *
 *   rows    : 0 <= rows < 2^31; LOOM_ERR_RANGE also when the grid would     *
 *             reach 2^32 work-items, as loom_launch_config_invoke reports   *
 *             for (rows, k, batch): only at 2^26 rows or more               *
 *   k       : elements per row, k % 4 == 0 (LOOM_ERR_SHAPE), 0 <= k <=      *
 *             131068 so |acc| <= 2^31 - 1 (LOOM_ERR_RANGE)                  *
 *   batch   : 1 <= batch <= 64 (LOOM_ERR_RANGE)                             *
 *   out     : f32[rows][batch], device                                      *
 *   acc     : int32[rows][batch], device, or NULL (not written)             *
 * ------------------------------------------------------------------------ */
int loom_i8_dequant_dot(const int32_t *w, const float *w_scale, const int32_t *x,
                        const float *x_scale, int64_t rows, int64_t k, int64_t batch,
                        float *out, int32_t *acc, void *stream);

/* ------------------------------------------------------------------------ *
 * The pages' literal packed signed-byte dot recurrence (TUNE §Apply the     *
 * same controls to a packed dot product).  For every output o, starting     *
 * from initial[o] (0 if NULL), every record r < count, in record order:     *
 *     v_j = f32(signed byte j of fields[r][o]) * f32(scales[r][o])          *
 *     sum = sum + v_j * rhs[r][o mod streams][j]     for j = 0, 1, 2, 3     *
 * each product and sum a separate f32 rounding (no fused multiply-add), so  *
 * the result is the serial recurrence bit for bit.                          *
 *   fields  : int32[records][outputs], record-major (consecutive outputs    *
 *             contiguous), 4-byte aligned                                   *
 *   scales  : binary16 bit patterns [records][outputs], 2-byte aligned      *
 *   rhs     : f32[records][streams][4] activations, 16-byte aligned; the    *
 *             streams are shared by all outputs (output o reads o mod       *
 *             streams)                                                      *
 *   streams : 1 <= streams < 2^31                                           *
 *   initial : f32[outputs] or NULL                                          *
 *   records : records allocated; 0 <= count <= records, count < 2^31, and   *
 *             4 * records * outputs fits in an int64 (LOOM_ERR_RANGE)     *
 *   outputs : 0 <= outputs <= 255 * (2^31 - 1); LOOM_ERR_RANGE also when    *
 *             the grid would reach 2^32 work-items, as                      *
 *             loom_launch_config_invoke reports for (outputs, count,        *
 *             streams): past 2^32 - 256 outputs, or 2^34 - 1024 when        *
 *             streams divides 64                                            *
 *   out     : f32[outputs]                                                  *
 * ------------------------------------------------------------------------ */
int loom_packed_dot(const int32_t *fields, const uint16_t *scales, const float *rhs, int64_t streams,
                    const float *initial, int64_t records, int64_t count, int64_t outputs, float *out,
                    void *stream);

/* ------------------------------------------------------------------------ *
 * The pages' guarded ragged row sum (TUNE §Keep guards and inner loops in   *
 * the source, @guide.sum_guarded_rows).  For each lane l < 32, rows are      *
 * walked in order up to count rounded up to a multiple of 4; a row at or    *
 * beyond count contributes 0 and is not read; otherwise its partial is the  *
 * in-order f32 sum, from 0, of values[row][l][c] for c < columns, each      *
 * taken as 0 (and not read) when l >= active_lanes.  sums[l] is the in-order *
 * f32 sum of the partials, from 0 -- the serial recurrence bit for bit.     *
 *   values       : f32[rows_alloc][32][4], 16-byte aligned                  *
 *   rows_alloc   : 0 <= rows_alloc <= 2^26                                  *
 *   count        : 0 <= count <= rows_alloc (the padded row need not exist) *
 *   columns      : 0 <= columns <= 4                                        *
 *   active_lanes : 0 <= active_lanes <= 32                                  *
 *   sums         : f32[32]                                                  *
 * ------------------------------------------------------------------------ */
int loom_sum_guarded_rows(const float *values, int64_t rows_alloc, int64_t count, int64_t columns,
                          int64_t active_lanes, float *sums, void *stream);

/* ------------------------------------------------------------------------ *
 * Routed row combine (TUNE §Separate route and payload lookahead: a routed  *
 * MoE combine).  For token t and column c, routes i < routes in order:      *
 *     id = ids[t][i]; if (uint32)id < num_rows:                             *
 *         acc[c] = acc[c] + weights[t][i] * payload[id][c]                  *
 * (product rounded, then added; acc starts at 0); out[t][c] = acc[c].  A   *
 * route whose id is outside [0, num_rows) is missing: neither its weight    *
 * nor its payload row is read.                                              *
 *   ids     : int32[tokens][routes]                                         *
 *   weights : f32[tokens][routes]                                           *
 *   payload : f32[num_rows][hidden] expert-output rows, 16-byte aligned     *
 *   num_rows: 0 <= num_rows < 2^31                                          *
 *   tokens  : 0 <= tokens < 2^31; routes, hidden: 0 .. 2^20                 *
 *   hidden  : a multiple of 4 (LOOM_ERR_SHAPE otherwise)                    *
 *   out     : f32[tokens][hidden], 16-byte aligned                          *
 * ------------------------------------------------------------------------ */
int loom_routed_combine(const int32_t *ids, const float *weights, const float *payload, int64_t num_rows,
                        int64_t tokens, int64_t routes, int64_t hidden, float *out, void *stream);

/* ------------------------------------------------------------------------ *
 * The int8 feed-forward operators.  Activations are quantised by token       *
 * (loom_quantize_rows), multiplied by int8 weights with one scale a channel, *
 * for any number of tokens, and every result is in token order.             *
 * ------------------------------------------------------------------------ */

/* Element types of activations, outputs and gradients. */
typedef enum loom_type { LOOM_F32 = 0, LOOM_F16 = 1, LOOM_BF16 = 2 } loom_type;

/* Activations of a gated unit: g / (1 + exp(-g)); g Phi(g) (erf); its tanh
 * form 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))); max(g, 0). */
typedef enum loom_activation { LOOM_SILU = 0, LOOM_GELU = 1, LOOM_GELU_TANH = 2, LOOM_RELU = 3 } loom_activation;

/* ------------------------------------------------------------------------ *
 * Symmetric int8 quantisation of rows (tokens).  With a = max_c |x[r][c]|:  *
 *     scale[r] = a / 127,   q[r][c] = rint(x[r][c] * (127 / a))             *
 * each quotient and product one f32 rounding, rint to even.  A row with     *
 * a < 2^-119 (an empty or zero row too) gives zeros and scale 0; a row that *
 * holds an infinity or a NaN gives zeros and scale NaN, which makes every   *
 * product of that row NaN.                                                  *
 *   x          : type[rows], rows row_stride elements apart, device,        *
 *                aligned to its element                                     *
 *   rows, cols : 0 .. 2^31 - 1; cols % 4 == 0 (LOOM_ERR_SHAPE)              *
 *   row_stride : >= cols (LOOM_ERR_SHAPE); 4 * rows * row_stride must fit   *
 *                in an int64 (LOOM_ERR_RANGE)                               *
 *   q          : int32[rows][cols/4] packed int8, device                    *
 *   scale      : f32[rows], device                                          *
 * ------------------------------------------------------------------------ */
int loom_quantize_rows(const void *x, int type, int64_t rows, int64_t cols, int64_t row_stride, int32_t *q,
                       float *scale, void *stream);

/* ------------------------------------------------------------------------ *
 * Int8 matrix product with a scale for each token and each channel.         *
 *     acc[t][n] = sum_{i < k} w[n][i] * x[t][i]            (exact, int32)   *
 *     out[t][n] = (f32(acc[t][n]) * w_scale[n]) * x_scale[t] + bias[n]      *
 * each operation one f32 rounding, the result rounded once to the output    *
 * type; a NULL x_scale or bias leaves its operation out.                    *
 *   w          : int32[rows][k/4] packed int8 weights, device               *
 *   w_scale    : f32[rows], device                                          *
 *   x          : int32[tokens][k/4] packed int8 activations, device         *
 *   x_scale    : f32[tokens], device, or NULL (= 1)                         *
 *   bias       : f32[rows], device, or NULL (= 0)                           *
 *   rows       : channels, 0 <= rows < 2^31                                 *
 *   k          : k % 4 == 0 (LOOM_ERR_SHAPE), 0 <= k <= 131068              *
 *   tokens     : 0 <= tokens < 2^31; LOOM_ERR_RANGE also when the grid      *
 *                would reach 2^32 work-items, as loom_launch_config_invoke  *
 *                reports for (rows, k, tokens)                              *
 *   out        : type[tokens], rows out_stride >= rows elements apart       *
 *                (LOOM_ERR_SHAPE), device, aligned to its element;          *
 *                4 * tokens * out_stride must fit in an int64               *
 * ------------------------------------------------------------------------ */
int loom_i8_matmul(const int32_t *w, const float *w_scale, const int32_t *x, const float *x_scale, const float *bias,
                   int64_t rows, int64_t k, int64_t tokens, void *out, int type, int64_t out_stride, void *stream);

/* ------------------------------------------------------------------------ *
 * Gated projection: both products, the activation and the product of the    *
 * two in one kernel.  With g and u the scaled products of loom_i8_matmul    *
 * (no bias) for the two weights,                                            *
 *     out[t][n] = act(g[t][n]) * u[t][n]                                    *
 * in f32, rounded once to the output type.  Arguments as there, each for    *
 * both weights; act is a loom_activation, anything else LOOM_ERR_RANGE.      *
 * ------------------------------------------------------------------------ */
int loom_i8_gated_projection(const int32_t *w_gate, const float *gate_scale, const int32_t *w_up,
                             const float *up_scale, const int32_t *x, const float *x_scale, int64_t rows, int64_t k,
                             int64_t tokens, int act, void *out, int type, int64_t out_stride, void *stream);

/* ------------------------------------------------------------------------ *
 * Gradients of the gated projection, for tuning over frozen int8 weights.   *
 * With g, u recomputed (the same bits as the forward pass) and d = d_out,   *
 *     dg = d * u * act'(g),   du = d * act(g)                               *
 *     d_x[t][i] = sum_f dg[t][f] gate_scale[f] w_gate[f][i]                 *
 *                     + du[t][f] up_scale[f] w_up[f][i]                     *
 *     d_gate_scale[f] = sum_t dg[t][f] acc_gate[t][f] x_scale[t]            *
 *     d_up_scale[f]   = sum_t du[t][f] acc_up[t][f] x_scale[t]              *
 * d_x is the gradient of the dequantised activation x * x_scale, what a     *
 * straight-through estimator passes on.  ReLU's derivative at 0 is 0.  All  *
 * sums are f32 in a fixed order: the same bits on every call.  d_x is a     *
 * product of the weights and the coefficients dg gate_scale, du up_scale,   *
 * which are whole for f32 gradients, rounded to at least 16 bits for f16    *
 * ones and to 11 bits for bf16 ones (there by at most 2^-30 of the token's  *
 * largest coefficient where that is more), and d_x is then rounded once.    *
 *   d_out        : type[tokens], rows d_stride >= rows elements apart       *
 *   d_x          : type[tokens][k] (the type of d_out), device, or NULL     *
 *   d_gate_scale, d_up_scale : f32[rows], device, or NULL                   *
 *   workspace    : device memory, 16-byte aligned, of at least the bytes    *
 *                  that loom_i8_gated_projection_backward_workspace gives   *
 *                  for the same sizes (LOOM_ERR_RANGE); its contents after  *
 *                  the call mean nothing                                    *
 *   rows         : 0 <= rows <= 2^21 (LOOM_ERR_RANGE)                     *
 * With no tokens the scale gradients are 0, with no channels d_x is.        *
 * ------------------------------------------------------------------------ */
int loom_i8_gated_projection_backward_workspace(int64_t rows, int64_t k, int64_t tokens, int type, int64_t *bytes);
int loom_i8_gated_projection_backward(const int32_t *w_gate, const float *gate_scale, const int32_t *w_up,
                                      const float *up_scale, const int32_t *x, const float *x_scale, int64_t rows,
                                      int64_t k, int64_t tokens, int act, const void *d_out, int type,
                                      int64_t d_stride, void *d_x, float *d_gate_scale, float *d_up_scale,
                                      void *workspace, int64_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------ *
 * A layer of experts with 4-bit weights.  loom_route_experts chooses each    *
 * token's experts, loom_group_routes puts the routes in the order of their   *
 * experts, the loom_i4_expert_ products take each expert's rows together, and *
 * loom_routed_combine (its ids the slots, its payload the last product's     *
 * rows) brings them back to the tokens.                                      *
 * ------------------------------------------------------------------------ */

/* Scores of experts: exp(l) / sum exp(l) over a token's experts; 1 / (1 + exp(-l)). */
typedef enum loom_score { LOOM_SOFTMAX = 0, LOOM_SIGMOID = 1 } loom_score;

/* ------------------------------------------------------------------------ *
 * Routing of tokens to experts.  With l a token's logits, s their scores    *
 * and c the choices, s + bias or, without a bias, l:                        *
 *  - the experts are `groups` runs of experts / groups neighbours; a group's *
 *    value is its largest choice (group_top 1), or the sum of its two largest *
 *    (group_top 2; without a bias, of its two largest scores).  Only the     *
 *    top_groups groups of the largest values stay.                          *
 *  - ids: the top_k experts of the largest choices among them, falling; ties *
 *    go to the lower group and the lower expert.                            *
 *  - weights: scale * s[ids], or scale * s[ids] / sum s[ids] where           *
 *    renormalize is not 0 (the bias only chooses).                          *
 * An expert whose logit or choice is -infinity is never chosen; where fewer  *
 * than top_k are left, the rest of ids is -1 with weight 0 (a missing route  *
 * of loom_group_routes and loom_routed_combine).  A token that has a NaN or  *
 * +infinity among its logits, or a NaN among the choices of experts whose    *
 * logit is not -infinity, gets ids 0 .. top_k - 1 and weights NaN.           *
 * Choices that are computed are computed and compared in 64 bits, weights    *
 * in f32; a ratio of renormalised weights stays exact where the scores       *
 * themselves vanish.                                                        *
 *   logits     : type[tokens], rows row_stride >= experts elements apart     *
 *                (LOOM_ERR_SHAPE), device, aligned to its element           *
 *   tokens     : 0 .. 2^31 - 1; 4 * tokens * row_stride must fit in an int64 *
 *   experts    : 1 .. 1024; groups: 1 .. 64, a divisor of experts            *
 *                (LOOM_ERR_SHAPE); top_groups: 1 .. groups                  *
 *   top_k      : 1 .. 64, at most top_groups * experts / groups              *
 *                (LOOM_ERR_SHAPE)                                           *
 *   bias       : f32[experts], device, or NULL                              *
 *   ids        : int32[tokens][top_k]; weights : f32[tokens][top_k]          *
 * ------------------------------------------------------------------------ */
int loom_route_experts(const void *logits, int type, int64_t tokens, int64_t experts, int64_t row_stride, int score,
                       const float *bias, int64_t groups, int64_t top_groups, int64_t group_top, int64_t top_k,
                       int renormalize, float scale, int32_t *ids, float *weights, void *stream);

/* ------------------------------------------------------------------------ *
 * Gradient of the routing weights with respect to the logits, the choice     *
 * held.  With d = scale * d_weights over a token's routes i, at their experts: *
 *     softmax:      d_l[j] = s_j (d_j - sum_i s_i d_i), d_j = 0 elsewhere    *
 *     sigmoid:      d_l[i] = d_i s_i (1 - s_i)                               *
 *     renormalised, w_i = s_i / sum s: d_l[i] = w_i (d_i - sum_j w_j d_j),   *
 *                   for a sigmoid times 1 - s_i                             *
 * in f32, rounded once to the type of the logits; every other d_l is 0.  A   *
 * route whose id is outside [0, experts) takes no part (and its d_weights is *
 * not read); an expert that is named twice takes the sum of its terms in     *
 * route order.  A token without routes gets zeros.                          *
 *   logits, ids, d_weights : as there, the logits of the forward pass        *
 *   d_logits   : type[tokens], rows d_stride >= experts elements apart       *
 * ------------------------------------------------------------------------ */
int loom_route_experts_backward(const void *logits, int type, int64_t tokens, int64_t experts, int64_t row_stride,
                                int score, int64_t top_k, int renormalize, float scale, const int32_t *ids,
                                const float *d_weights, void *d_logits, int64_t d_stride, void *stream);

/* ------------------------------------------------------------------------ *
 * Routes in the order of their experts.  Route p = token * routes + i leads  *
 * to expert ids[p]; the routes of one expert keep their order.               *
 *     slots[p]   = the place of route p, or -1 where ids[p] is no expert     *
 *     rows[at]   = the token of the route at that place, -1 past the last    *
 *     offsets[e] = the first place of expert e; offsets[experts] = how many  *
 *   ids       : int32[tokens][routes], device                               *
 *   tokens, routes : tokens * routes < 2^31, routes <= 2^20                  *
 *   experts   : 1 .. 1024                                                   *
 *   slots, rows : int32[tokens * routes]; offsets : int32[experts + 1]       *
 *               (written also where there are no tokens)                    *
 *   workspace : device memory, 4-byte aligned, of at least the bytes that    *
 *               loom_group_routes_workspace gives for the same sizes         *
 *               (LOOM_ERR_RANGE; it may be NULL where that is 0)            *
 * ------------------------------------------------------------------------ */
int loom_group_routes_workspace(int64_t tokens, int64_t routes, int64_t experts, int64_t *bytes);
int loom_group_routes(const int32_t *ids, int64_t tokens, int64_t routes, int64_t experts, int32_t *slots, int32_t *rows,
                      int32_t *offsets, void *workspace, int64_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------ *
 * Matrix product of int8 activations with 4-bit weights that have a scale    *
 * for each channel and group of k.                                          *
 *     acc[t][n][g] = sum of w[n][i] * x[t][i] over group g     (exact, int32) *
 *     out[t][n] = (sum_g scale[n][g] * f32(acc[t][n][g])) * x_scale[t] + bias[n] *
 * in f32 (the sum over groups in a fixed order), rounded once to the output  *
 * type; a NULL x_scale or bias leaves its operation out.  A group longer than *
 * 128 is the f32 sum of its parts of 128, each of which is exact.  Sums      *
 * before x_scale are held 16 times as large: from 2^124 on they overflow.    *
 * Packed 4-bit weights: two's complement, 32 neighbours of k in 16 bytes;    *
 * byte b of them holds element b in its low four bits and element 16 + b in  *
 * its high four.                                                            *
 *   w          : int32[rows][k/8], device, 16-byte aligned                  *
 *   w_scale    : scale_type[rows][ceil(k / group)], device                  *
 *   scale_type : a loom_type                                                *
 *   group      : a power of two (LOOM_ERR_SHAPE), 32 .. 2^17 (LOOM_ERR_RANGE); *
 *                a last group may be shorter, one of k or more is one scale  *
 *                a channel                                                  *
 *   x          : int32[tokens][k/4] packed int8 activations, device,         *
 *                16-byte aligned                                            *
 *   x_scale    : f32[tokens], device, or NULL (= 1)                         *
 *   bias       : f32[rows], device, or NULL (= 0)                           *
 *   rows       : channels, 0 <= rows < 2^31                                 *
 *   k          : k % 32 == 0 (LOOM_ERR_SHAPE), 0 <= k <= 131040             *
 *   tokens     : 0 <= tokens < 2^31; LOOM_ERR_RANGE also when the grid      *
 *                would reach 2^32 work-items, as loom_launch_config_invoke  *
 *                reports for (rows, k, tokens, group)                       *
 *   out        : type[tokens], rows out_stride >= rows elements apart       *
 *                (LOOM_ERR_SHAPE), device, aligned to its element;          *
 *                4 * tokens * out_stride must fit in an int64               *
 * ------------------------------------------------------------------------ */
int loom_i4_matmul(const int32_t *w, const void *w_scale, int scale_type, int64_t group, const int32_t *x,
                   const float *x_scale, const float *bias, int64_t rows, int64_t k, int64_t tokens, void *out,
                   int type, int64_t out_stride, void *stream);

/* ------------------------------------------------------------------------ *
 * The same product for experts: routed row p, offsets[e] <= p <              *
 * offsets[e + 1], is row index[p] of x times the weights of expert e.        *
 *     out[p][n] = loom_i4_matmul's for w[e], w_scale[e], bias[e], x[index[p]] *
 * Rows of out that belong to no expert are left as they were.  offsets may   *
 * name any rows: only those within [0, pairs) count, and an expert whose     *
 * offsets fall has none.  Where ranges of experts overlap, no row of any     *
 * expert has a defined value, and each may be left as it was.  A row whose   *
 * index is outside [0, x_rows) becomes NaN.                                 *
 *   w          : int32[experts][rows][k/8], w_scale : scale_type[experts]    *
 *                [rows][ceil(k / group)], bias : f32[experts][rows] or NULL   *
 *   x          : int32[x_rows][k/4], x_scale : f32[x_rows] or NULL           *
 *   index      : int32[pairs], device, or NULL (row p of x)                 *
 *   x_rows     : at least 1, and pairs without an index (LOOM_ERR_SHAPE)     *
 *   offsets    : int32[experts + 1], device                                 *
 *   experts    : 1 .. 1024                                                  *
 *   pairs      : routed rows, 0 <= pairs < 2^31, and the grid as above, of   *
 *                (rows, k, pairs, group, experts)                           *
 *   out        : type[pairs], rows out_stride apart                         *
 * ------------------------------------------------------------------------ */
int loom_i4_expert_matmul(const int32_t *w, const void *w_scale, int scale_type, int64_t group, const int32_t *x,
                          const float *x_scale, int64_t x_rows, const int32_t *index, const int32_t *offsets,
                          const float *bias, int64_t experts, int64_t rows, int64_t k, int64_t pairs, void *out,
                          int type, int64_t out_stride, void *stream);

/* Gated projection of experts: act(g) * u with g and u the products above (no
 * bias) for the two weights, in f32, rounded once.  act is a loom_activation,
 * anything else LOOM_ERR_RANGE. */
int loom_i4_expert_gated_projection(const int32_t *w_gate, const void *gate_scale, const int32_t *w_up,
                                    const void *up_scale, int scale_type, int64_t group, const int32_t *x,
                                    const float *x_scale, int64_t x_rows, const int32_t *index, const int32_t *offsets,
                                    int64_t experts, int64_t rows, int64_t k, int64_t pairs, int act, void *out,
                                    int type, int64_t out_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LOOM_H */
