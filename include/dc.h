/*
 * dc.h - C ABI of libdc.so, a data-parallel gradient-reduction path for one
 * MI355X (gfx950) GPU.
 *
 * W simulated data-parallel ranks are the rows of a [W, ld] gradient slab in
 * device memory (row r = rank r's gradient; row-major; `ld` = row stride in
 * elements).  Every device entry point enqueues work on the given HIP stream
 * and returns at once; its results are valid once that stream reaches them.
 *
 * Pages cited (by title and section):
 *   [DS] DeepSpeed issue "[REQUEST] DeepCompile ZeRO-1: reduce-to-owner
 *        instead of AllReduce"
 *   [MT] MaxText PR "Defer the data-parallel gradient all-reduce to update()
 *        under gradient accumulation"
 *   [AG] "AllGather" (collective-communication notes)
 *
 * Typical use:
 *   once per layout   dc_partition_ids, then dc_build_owner_map (device
 *                     tables); per bucket, dc_validate_tasks on the host
 *                     copy of its task table and a plan (dc_plan_flush on
 *                     the host, or dc_plan_flush_device)
 *   every step        per bucket, as its gradients are complete,
 *                     dc_flush_bucket_planned (dc_flush_bucket without a
 *                     plan; dc_flush_bucket_buffers[_planned] to read each
 *                     rank's own gradient buffers and write the grad buffers)
 *   under gradient    dc_accumulate for each micro-batch, then one
 *   accumulation      dc_deferred_reduce (or dc_accumulate_reduce for the
 *                     last micro-batch) ([MT] What)
 *   a layer's         dc_linear forward, dc_bias_act_backward and
 *   gradients         dc_linear_backward, whose weight gradient may go
 *                     straight into an accumulator row; dc_norm around a
 *                     block and dc_embedding before it, likewise with
 *                     dc_norm_backward and dc_embedding_backward
 *   clipping          dc_grad_clip on the reduced gradients (dc_grad_norm:
 *                     their global norm alone)
 *   the owner's step  dc_muon_update on the parameters whose reduced
 *                     gradient the owner holds whole (dc_orthogonalize: its
 *                     orthogonalisation alone)
 *   collectives       dc_reduce_scatter / dc_all_gather and their ring-order,
 *                     step-by-step and relaid (dc_relayout_bucket +
 *                     dc_reduce_scatter_v) forms
 *
 * Conventions shared by every function:
 *   - Return value: DC_OK (0) or one of the DC_ERR_* codes below.  Argument
 *     checks run on the host before anything is enqueued; a failed check
 *     enqueues nothing.  dc_last_error() gives a message for the calling
 *     thread's last failure.  No C++ exception crosses this boundary.
 *   - "device" pointers are HIP device (or managed) memory; "host" pointers
 *     are ordinary host memory read synchronously during the call.
 *   - The caller owns every buffer.  The library allocates nothing, keeps no
 *     pointer after the call returns (device pointers are used by the
 *     enqueued kernels until they finish) and never synchronizes the stream.
 *   - `stream` is a hipStream_t passed as void*; NULL is the default stream.
 *   - dtype: DC_BF16 (bfloat16 stored as uint16 bit patterns) or DC_F32.
 *   - Slab base pointers must be 16-byte aligned and `ld` a multiple of 16
 *     bytes (8 bf16 or 4 fp32 elements), else DC_ERR_ALIGN.
 *   - Row strides, column counts and byte counts above 2^44 are DC_ERR_SHAPE,
 *     so that no size computed from them can overflow int64.
 *   - Sums are folded in fp32 in ascending rank order (member order within a
 *     communicator), starting from the first contribution, and rounded once
 *     to the dtype (round to nearest even; NaN -> quiet NaN 0x7FC0|sign for
 *     bf16).  fp32 arithmetic keeps subnormals and is never contracted.
 */
#ifndef DC_H
#define DC_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t dc_status;

#define DC_OK 0
#define DC_ERR_NULL 1        /* a required pointer is NULL */
#define DC_ERR_ARG 2         /* a scalar argument is out of range, or buffers overlap */
#define DC_ERR_SHAPE 3       /* sizes or strides do not fit together */
#define DC_ERR_ALIGN 4       /* a slab base or stride is not 16-byte aligned */
#define DC_ERR_DTYPE 5       /* unknown dtype */
#define DC_ERR_TASKS 6       /* a task table breaks its contract (dc_validate_tasks) */
#define DC_ERR_HIP 7         /* a HIP launch or runtime call failed */
#define DC_ERR_UNSUPPORTED 8 /* a valid request this library does not handle */

#define DC_BF16 0
#define DC_F32 1

#define DC_ORDER_RANK 0
#define DC_ORDER_RING 1

#define DC_SCHED_RING 0      /* all-gather step schedules (dc_all_gather_step) */
#define DC_SCHED_BIDIR 1
#define DC_SCHED_RD 2

#define DC_ACT_NONE 0        /* activations of the linear layer */
#define DC_ACT_RELU 1
#define DC_ACT_GELU 2        /* v Phi(v), Phi the normal distribution's */
#define DC_ACT_SILU 3        /* v / (1 + exp(-v)) */

#define DC_PRODUCT_FORWARD 0 /* products of the linear layer */
#define DC_PRODUCT_DX 1
#define DC_PRODUCT_DW 2

#define DC_SCALE_NONE 0      /* shape factor of a matrix update: 1 */
#define DC_SCALE_ASPECT 1    /* sqrt(max(1, rows / cols)) */
#define DC_SCALE_RMS 2       /* 0.2 sqrt(max(rows, cols)) */
#define DC_HOLD_AUTO 0       /* what Newton-Schulz steps hold a value in: by the types */
#define DC_HOLD_ONE 1        /* one fp16 */
#define DC_HOLD_PAIR 2       /* a pair of fp16 */
#define DC_NS_MAX_STEPS 16   /* Newton-Schulz steps per call */

#define DC_MAX_W 64          /* simulated ranks per slab */
#define DC_MAX_GROUPS 64     /* parameter groups per owner map */
#define DC_MAX_COMMS 8       /* communicators per flush */

/* One bucket entry: a whole parameter's gradient ([DS] "Describe
 * alternatives": buckets hold one full-parameter task each, in gradient
 * arrival order).  32 bytes.
 *   offset   first column of the task, relative to the bucket's first column
 *   numel    columns of the task (>= 0)
 *   param    index into the owner map
 *   comm     index into the flush's communicator table
 * For the slab flushes a bucket's table is sorted and packed: offset[0] = 0,
 * offset[t+1] = offset[t] + numel[t], and the numels sum to the bucket size.
 * dc_flush_bucket_buffers takes sorted, disjoint tasks with gaps allowed (its
 * offsets are coordinates only) and does not read `param`.  `reserved` is
 * not read by any entry point. */
typedef struct {
  int64_t offset;
  int64_t numel;
  int32_t param;
  int32_t comm;
  int64_t reserved;
} dc_task;

/* A communicator over the W ranks ([DS] Design points, groups reduced over a
 * different communicator, e.g. MoE experts): `size` c divides W and the ranks
 * split into W/c blocks; block b's members are {b*c + i} when stride == 1,
 * or {b + i*W/c} when stride == W/c (i = 0..c-1).  Entry 0 of every table is
 * the data-parallel communicator {W, 1}. */
typedef struct {
  int32_t size;
  int32_t stride;
} dc_comm;

/* Probe record of one flush ([DS] problem statement, the probe report, and
 * "reduce_probe").  Per rank r: written[r] = elements the flush writes to row
 * r, kept[r] = elements of tasks whose parameter rank r holds (its partition
 * appears in the parameter's partition list), discarded[r] = written - kept. */
typedef struct {
  int32_t tasks;
  int32_t owner_tasks;
  int32_t pre_div;
  int32_t dtype;
  int64_t reduced_elems;
  int64_t owner_elems;
  int64_t written[DC_MAX_W];
  int64_t kept[DC_MAX_W];
  int64_t discarded[DC_MAX_W];
} dc_probe;

/* One piece of a bucket relayout: bucket columns [src, src+len) move to
 * relaid columns [dst, dst+len).  32 bytes. */
typedef struct {
  int64_t src;
  int64_t dst;
  int64_t len;
  int64_t reserved;
} dc_piece;

/* One tile record of a planned bucket flush (dc_plan_flush).  The planned
 * flush cuts a bucket into plan tiles of 64 consecutive 16-byte column
 * vectors (1 KiB of each row; tile b of a bucket starting at column c covers
 * the row's vectors [v0 + 64 b, v0 + 64 (b + 1)), v0 = floor(c / E / 64) * 64
 * with E elements per vector, clipped to the bucket's last vector), one
 * workgroup per tile, and this record says which tasks a tile overlaps and,
 * when the whole tile lies inside one task and the bucket, which rows
 * receive its sums.  16 bytes.  A plan of n records keeps them XCD-major, in
 * the order the 8 XCDs run the tiles: the record of tile b sits at index
 * (b mod 8) floor(n/8) + min(b mod 8, n mod 8) + floor(b/8).
 *   first, last   indices of the first and last task overlapping the tile
 *                 (last < first: none)
 *   root          whole tile inside one task: the row that alone receives
 *                 the sums (the owner, or under ZeRO-2 the partition's rank),
 *                 or -1 for every member of each block (AllReduce)
 *   flags         bit 0: the whole tile lies inside task `first` and the
 *                 bucket; bits 8..15: that task's communicator */
typedef struct {
  int32_t first;
  int32_t last;
  int32_t root;
  int32_t flags;
} dc_tile;

/* One matrix of dc_orthogonalize or dc_muon_update: rows x cols, row-major.
 * 48 bytes.
 *   grad, ld_grad  device, the gradient: row r starts at grad + r * ld_grad
 *                  (in elements; any alignment), ld_grad >= cols
 *   out, ld_out    device, the result, or the weights that are updated
 *   momentum       device fp32 [rows][cols], read and written by
 *                  dc_muon_update; not used by dc_orthogonalize
 *   rows, cols     at least 1 */
typedef struct {
  const void* grad;
  void* out;
  float* momentum;
  int64_t ld_grad;
  int64_t ld_out;
  int32_t rows;
  int32_t cols;
} dc_matrix;

/* One gradient of dc_grad_norm or dc_grad_clip: rows x cols, row-major, in any
 * order of rows.  64 bytes.
 *   grad, ld_grad  device: row r starts at grad + r * ld_grad (in elements; any
 *                  alignment to an element), ld_grad >= cols
 *   out, ld_out    device, dc_grad_clip's result; may be grad (same ld)
 *   rows, cols     at least 0
 *   counted        the first rows, 0 to rows, that the norm counts: 1 for a
 *                  reduced gradient that every rank's row holds
 *   dtype          DC_BF16 or DC_F32, of grad and out
 *   reserved       not read */
typedef struct {
  const void* grad;
  void* out;
  int64_t ld_grad;
  int64_t ld_out;
  int64_t rows;
  int64_t cols;
  int64_t counted;
  int32_t dtype;
  int32_t reserved;
} dc_gradient;

/* Library version string (static storage). */
const char* dc_version(void);

/* Static description of a status code. */
const char* dc_strerror(dc_status status);

/* Message of the calling thread's last failed call ("" if none). */
const char* dc_last_error(void);

/* Partition lists ([DS] Design points, the owner map: the ZeRO
 * optimizer's param_to_partition_ids lists every optimizer partition holding
 * a piece of a parameter).  For each group g, the params
 * group_begin[g] .. group_begin[g+1]-1 are laid end to end in declaration
 * order (flat offset a_i = sum of earlier sizes in the group); the group's
 * T_g elements split into group_parts[g] equal partitions of
 * S_g = ceil(T_g / group_parts[g]) elements (the last one shorter); a
 * non-empty param's list is floor(a_i/S_g) .. floor((a_i+n_i-1)/S_g), an
 * empty param's list is empty.
 *   numel         device int64[num_params], each in [0, 2^48)
 *   group_begin   host int32[num_groups+1], non-decreasing, 0 .. num_params
 *   group_parts   host int32[num_groups], each in [1, DC_MAX_W]
 *   flat_offset   device int64[num_params] out: a_i
 *   part_size     device int64[num_groups] out: S_g
 *   pid_offsets   device int32[num_params+1] out: CSR row starts
 *   pids          device int32[pids_capacity] out: CSR entries
 * pids_capacity must be at least num_params + sum_g (group_parts[g] - 1),
 * the largest count any sizes can produce, else DC_ERR_SHAPE.  Sizes outside
 * [0, 2^48) are not checked on the host; the kernel treats a negative size
 * as 0.  One workgroup scans all groups. */
dc_status dc_partition_ids(int32_t W, int32_t num_params, const int64_t* numel,
                           int32_t num_groups, const int32_t* group_begin,
                           const int32_t* group_parts, int64_t* flat_offset, int64_t* part_size,
                           int32_t* pid_offsets, int32_t* pids, int64_t pids_capacity,
                           void* stream);

/* Owner map ([DS] Design points): a param whose partition list has a
 * single element is held by one rank only and gets that rank as its owner; a
 * param listed in two or more partitions (it straddles a partition
 * boundary) or in none gets -1, meaning AllReduce.  A group takes part only when its communicator is the
 * data-parallel one: group_comm_size[g] == W and group rank i maps to global
 * rank i for every i; every param of another group gets -1.
 *   pid_offsets, pids      device CSR from dc_partition_ids; pids_capacity is
 *                          the length of pids (entries beyond it are not read)
 *   group_begin            host int32[num_groups+1] (as for dc_partition_ids)
 *   group_comm_size        host int32[num_groups]
 *   group_rank_to_global   host int32[num_groups * W], row g = group g's
 *                          group rank -> global rank map (pad with -1)
 *   owner                  device int32[num_params] out
 *   counts                 device int32[2*num_groups] out: counts[2g] = params
 *                          with an owner, counts[2g+1] = params with two or
 *                          more entries (at most group_parts[g]-1)
 * Entries of pids outside [0, W) are reported as no owner. */
dc_status dc_build_owner_map(int32_t W, int32_t num_params, const int32_t* pid_offsets,
                             const int32_t* pids, int64_t pids_capacity, int32_t num_groups,
                             const int32_t* group_begin,
                             const int32_t* group_comm_size, const int32_t* group_rank_to_global,
                             int32_t* owner, int32_t* counts, void* stream);

/* Host check of a bucket's task table (run once when the bucket layout is
 * built): sorted and packed from offset 0, numel >= 0 summing to
 * bucket_numel, param in [0, num_params), comm in [0, num_comms); comms[0] is
 * {W, 1} and every comm's size divides W with stride 1 or W/size.
 * tasks and comms are host arrays.  Returns DC_ERR_TASKS with a message
 * naming the first broken entry. */
dc_status dc_validate_tasks(int32_t W, const dc_task* tasks, int32_t num_tasks,
                            int64_t bucket_numel, int32_t num_params, const dc_comm* comms,
                            int32_t num_comms);

/* Bucket flush ([DS] problem statement and "Describe the solution").
 * For every task t, column j of the bucket inside t, and block of the task's
 * communicator (c members m_0 < ... < m_{c-1}):
 *   v_k = pre_div ? round_dtype(fp32(x[m_k][j]) / c) : x[m_k][j]
 *   y   = round_dtype(((v_0 + v_1) + ...) + v_{c-1})      (fp32)
 * A task on comm 0 whose param has owner o >= 0 writes y to row o only (the
 * reduce-to-owner branch: same sum, same operand order, one destination);
 * every other task writes y to every member of the block (AllReduce).
 * owner == NULL is the empty map: every task AllReduces, bit for bit the path
 * without owners ([DS] Design points, "No native flag").  Elements the flush
 * does not write keep their contents.
 *   slab_in, ld_in     device [W, ld_in] gradients (bf16 or fp32 per dtype)
 *   slab_out, ld_out   device [W, ld_out] results; may equal slab_in (same
 *                      ld) for an in-place flush; partial overlap is DC_ERR_ARG
 *   bucket_col         first slab column of the bucket
 *   bucket_numel       columns of the bucket; bucket_col + bucket_numel must
 *                      not exceed ld_in or ld_out
 *   tasks, num_tasks   device dc_task[num_tasks] (see dc_validate_tasks)
 *   owner, num_params  device int32[num_params] from dc_build_owner_map, or NULL
 *   comms, num_comms   host dc_comm[num_comms], 1 <= num_comms <= DC_MAX_COMMS
 *   pre_div            0 or 1
 * The task table is read on the device and is not checked here (validate it
 * once with dc_validate_tasks).  A table that breaks the contract still
 * never makes the kernel touch memory outside the bucket's columns of the
 * two slabs: an out-of-range param or owner entry means AllReduce, an
 * out-of-range comm means comm 0, and columns no task covers are not
 * written. */
dc_status dc_flush_bucket(int32_t W, int32_t dtype, const void* slab_in, int64_t ld_in,
                          void* slab_out, int64_t ld_out, int64_t bucket_col,
                          int64_t bucket_numel, const dc_task* tasks, int32_t num_tasks,
                          const int32_t* owner, int32_t num_params, const dc_comm* comms,
                          int32_t num_comms, int32_t pre_div, void* stream);

/* ZeRO-2 owner path ([DS] "Follow-up": ZeRO-2 keeps real per-rank buffers at
 * offsets, so the reduce-to-owner optimization extends to every piece of a
 * parameter).  Same fold as dc_flush_bucket, but on the data-parallel comm
 * (comm 0) every element goes to the rank whose optimizer partition holds it:
 * element e of a task of param i sits at flat position flat_offset[i] + e of
 * its group and belongs to partition floor((flat_offset[i] + e) /
 * part_size[i]); the sum is written to that row only.  A task whose param has
 * part_size 0 (a group on another communicator), or any task on another
 * comm, AllReduces within its blocks as in dc_flush_bucket.
 *   flat_offset   device int64[num_params]: dc_partition_ids' flat offsets
 *   part_size     device int64[num_params]: S of the param's group, or 0
 * Other arguments, checks and guarantees as in dc_flush_bucket (a partition
 * index outside [0, W) means AllReduce for that element). */
dc_status dc_flush_bucket_zero2(int32_t W, int32_t dtype, const void* slab_in, int64_t ld_in,
                                void* slab_out, int64_t ld_out, int64_t bucket_col,
                                int64_t bucket_numel, const dc_task* tasks, int32_t num_tasks,
                                const int64_t* flat_offset, const int64_t* part_size,
                                int32_t num_params, const dc_comm* comms, int32_t num_comms,
                                int32_t pre_div, void* stream);

/* Plan of a bucket flush ([DS] Design points: the roots of a bucket's
 * collectives are computed for the whole bucket before any reduction).
 * Host only, once per bucket layout: for every plan tile (see dc_tile) over
 * columns [bucket_col, bucket_col + bucket_numel), the tasks it overlaps
 * and, for a tile inside one task, the rows its sums go to:
 *   owner-map mode (flat_offset == NULL): the owner owner[param] of a task on
 *   comm 0 when owner is given and the entry lies in [0, W), else -1;
 *   ZeRO-2 mode (flat_offset and part_size given, owner NULL): for a task on
 *   comm 0 whose param has part_size S > 0, the partition
 *   floor((flat_offset[param] + e) / S) when every element e of the tile
 *   lies in the same one inside [0, W) (otherwise the tile is not whole),
 *   else -1.
 *   tasks, num_tasks      host dc_task[num_tasks]; must pass dc_validate_tasks
 *                         (else DC_ERR_TASKS)
 *   owner                 host int32[num_params] or NULL
 *   flat_offset, part_size host int64[num_params] or NULL (ZeRO-2)
 *   comms, num_comms      host, as for dc_flush_bucket
 *   tiles, capacity       host dc_tile[capacity] out; NULL asks for the count
 *   num_tiles             out: the tile count, a function of dtype,
 *                         bucket_col and bucket_numel only
 *   root_tiles            out (may be NULL): tiles whose sums go to one row
 *                         (whole tiles with root >= 0), set with the tiles
 * Fewer than *num_tiles slots is DC_ERR_SHAPE.  The plan stays valid while
 * the layout, owner map (or partition sizes) and dtype stay the same. */
dc_status dc_plan_flush(int32_t W, int32_t dtype, int64_t bucket_col, int64_t bucket_numel,
                        const dc_task* tasks, int32_t num_tasks, const int32_t* owner,
                        const int64_t* flat_offset, const int64_t* part_size, int32_t num_params,
                        const dc_comm* comms, int32_t num_comms, dc_tile* tiles,
                        int64_t capacity, int64_t* num_tiles, int64_t* root_tiles);

/* The plan of dc_plan_flush computed on the device ([DS] Design points: a
 * bucket's reduction destinations are settled for the whole bucket before
 * it is reduced), for callers whose task table and owner map (or ZeRO-2
 * partition sizes) live in device memory: no host copy and no
 * synchronization.  The records are those dc_plan_flush writes for the same
 * arguments, bit for bit, and serve dc_flush_bucket_planned the same way.
 * One thread per tile binary-searches the task offsets.
 *   tasks                 device dc_task[num_tasks]; must be a table that
 *                         passes dc_validate_tasks (not checked here: another
 *                         table gives other records, and its params and
 *                         communicators index owner, flat_offset and
 *                         part_size only inside [0, num_params) and
 *                         [0, num_comms))
 *   owner                 device int32[num_params] or NULL (owner-map mode)
 *   flat_offset, part_size device int64[num_params] or NULL (ZeRO-2, as for
 *                         dc_plan_flush)
 *   comms, num_comms      host, as for dc_flush_bucket (checked)
 *   tiles, capacity       device dc_tile[capacity] out; NULL asks for the
 *                         count only (nothing is launched)
 *   num_tiles             host out: the tile count (as dc_plan_flush's)
 *   root_tiles            device int64 out, or NULL: set on the stream to
 *                         the count dc_plan_flush reports as root_tiles
 *                         (whole tiles with root >= 0); a caller that does
 *                         not read it back may pass num_tiles for
 *                         reduce-to-owner or ZeRO-2 buckets and 0 otherwise to
 *                         dc_flush_bucket_planned, which uses it only to pick
 *                         the launch shape
 * Fewer than *num_tiles slots is DC_ERR_SHAPE.  Stream-ordered: the plan is
 * ready for a planned flush later on the same stream. */
dc_status dc_plan_flush_device(int32_t W, int32_t dtype, int64_t bucket_col, int64_t bucket_numel,
                               const dc_task* tasks, int32_t num_tasks, const int32_t* owner,
                               const int64_t* flat_offset, const int64_t* part_size,
                               int32_t num_params, const dc_comm* comms, int32_t num_comms,
                               dc_tile* tiles, int64_t capacity, int64_t* num_tiles,
                               int64_t* root_tiles, void* stream);

/* Bucket flush with a plan (dc_plan_flush): the same results, bit for bit,
 * as dc_flush_bucket (flat_offset == NULL) or dc_flush_bucket_zero2
 * (flat_offset and part_size given, owner NULL) with the same arguments.  A
 * tile the plan marks whole streams its vectors with no search of the task
 * table and no staging; other tiles use the record's task range.  The
 * launch also keeps fewer workgroups resident per compute unit (it reserves
 * LDS it does not use): fewer, longer streams of loads in flight at once
 * measured faster for this access mix.
 *   tiles, num_tiles   device dc_tile[num_tiles] from dc_plan_flush for this
 *                      bucket, dtype, layout and map; num_tiles must equal
 *                      the planned count (else DC_ERR_SHAPE)
 *   root_tiles         the count dc_plan_flush reported, in [0, num_tiles]
 *                      (else DC_ERR_ARG); it only picks the residency cap:
 *                      buckets whose tiles mostly write one row keep more
 *                      workgroups per compute unit than those that write
 *                      every row, and any value gives the same results
 * Other arguments and checks as in dc_flush_bucket.  The plan is read on
 * the device and not checked: a stale or altered plan can give wrong sums,
 * and write columns of slab_out's rows outside the bucket but inside its
 * tile grid (the 64-vector tiles that cover the bucket), but never makes the
 * kernel touch memory outside the two slabs' W rows of ld columns (task
 * indices, roots and communicators are clamped to their ranges). */
dc_status dc_flush_bucket_planned(int32_t W, int32_t dtype, const void* slab_in, int64_t ld_in,
                                  void* slab_out, int64_t ld_out, int64_t bucket_col,
                                  int64_t bucket_numel, const dc_task* tasks, int32_t num_tasks,
                                  const int32_t* owner, const int64_t* flat_offset,
                                  const int64_t* part_size, int32_t num_params,
                                  const dc_comm* comms, int32_t num_comms, int32_t pre_div,
                                  const dc_tile* tiles, int64_t num_tiles, int64_t root_tiles,
                                  void* stream);

/* Bucket flush with copy-in and copy-out fused in ([DS] problem statement:
 * gradients enter the bucket from every rank and, after the reduction, the
 * copy-out moves the result into each rank's gradient buffer, skipping the
 * ranks whose buffer is empty; "Describe the solution": copy-out unchanged
 * and still correct).  No bucket is staged: rank r's gradient of task t is
 * read from in_ptrs[t*W + r] and the sum is written to out_ptrs[t*W + r]
 * for every member r of the block whose pointer is not NULL (a NULL pointer
 * is an empty buffer and is never written).  For every task t, element
 * e < numel and block of the task's communicator (members m_0 < ... < m_{c-1}):
 *   v_k = pre_div ? round_dtype(fp32(in_ptrs[t*W + m_k][e]) / c) : in_ptrs[t*W + m_k][e]
 *   y   = round_dtype(((v_0 + v_1) + ...) + v_{c-1})      (fp32)
 * the same values, in the same order, as dc_flush_bucket on a bucket filled
 * from those buffers; with exactly one non-NULL output (the owner) it is the
 * reduce-to-owner flush followed by the copy-out.
 *   bucket_numel       extent of the task coordinates: offsets and numel of
 *                      the tasks place them in [0, bucket_numel)
 *   tasks, num_tasks   device dc_task[num_tasks] sorted by offset, disjoint
 *                      (gaps allowed); param is not used; an out-of-range
 *                      comm means comm 0
 *   in_ptrs            device array [num_tasks * W] of device pointers, each
 *                      to numel elements of the dtype (rank r's gradient)
 *   out_ptrs           device array [num_tasks * W] of device pointers or NULL
 *   comms, num_comms   host dc_comm[num_comms] as in dc_flush_bucket
 *   pre_div            0 or 1
 * An output may be the same buffer as its own input (in place); otherwise
 * outputs must not overlap each other or any input (check the tables once
 * with dc_validate_buffer_tasks).  A task whose offset is a multiple of 16
 * bytes' worth of elements and whose pointers are all 16-byte aligned runs on
 * 16-byte vectors; any other element runs one at a time. */
dc_status dc_flush_bucket_buffers(int32_t W, int32_t dtype, int64_t bucket_numel,
                                  const dc_task* tasks, int32_t num_tasks,
                                  const void* const* in_ptrs, void* const* out_ptrs,
                                  const dc_comm* comms, int32_t num_comms, int32_t pre_div,
                                  void* stream);

/* Plan of a fused flush (dc_flush_bucket_buffers' tables), host only, once
 * per registration: the fused kernel cuts the bucket's coordinates
 * [0, bucket_numel) into tiles of 64 slots of 16 bytes (slot v covers
 * coordinates [v E, v E + E), E elements per 16 bytes), and tile b's record
 * names the first task starting at or before the tile and the last starting
 * inside it (last < first: none), and sets flags bit 0 when the tile's slots
 * all lie inside that one task, the task is on the data-parallel comm and its
 * offset is a multiple of E; root is -1.  Records are XCD-major as in
 * dc_tile.
 *   tasks, comms        host copies: tasks sorted, disjoint, inside the
 *                       bucket, comm in range (else DC_ERR_TASKS)
 *   tiles, capacity     host dc_tile[capacity] out; NULL asks for the count
 *   num_tiles           out: ceil(ceil(bucket_numel / E) / 64), 0 with no
 *                       tasks; fewer slots than that is DC_ERR_SHAPE */
dc_status dc_plan_flush_buffers(int32_t W, int32_t dtype, int64_t bucket_numel, const dc_task* tasks,
                                int32_t num_tasks, const dc_comm* comms, int32_t num_comms,
                                dc_tile* tiles, int64_t capacity, int64_t* num_tiles);

/* dc_plan_flush_buffers' records computed on the device, bit for bit, from a
 * task table in device memory (one thread per tile, binary search of the
 * task offsets): no host copy and no synchronization.
 *   tasks             device dc_task[num_tasks] in buffer coordinates; must
 *                     pass dc_validate_buffer_tasks (not checked here:
 *                     another table gives other records, every read and
 *                     write stays in the table and the plan)
 *   comms, num_comms  host, checked as for dc_plan_flush_buffers
 *   tiles, capacity   device dc_tile[capacity] out; NULL asks for the count
 *                     only (nothing is launched)
 *   num_tiles         host out: the tile count (dc_plan_flush_buffers')
 * Fewer than *num_tiles slots is DC_ERR_SHAPE.  Stream-ordered. */
dc_status dc_plan_flush_buffers_device(int32_t W, int32_t dtype, int64_t bucket_numel,
                                       const dc_task* tasks, int32_t num_tasks,
                                       const dc_comm* comms, int32_t num_comms, dc_tile* tiles,
                                       int64_t capacity, int64_t* num_tiles, void* stream);

/* dc_flush_bucket_buffers with a plan from dc_plan_flush_buffers: the same
 * results, bit for bit.  A tile the plan marks whole, whose task the kernel
 * finds covering the tile and whose W input and output pointers are 16-byte
 * aligned, streams from the task's pointer row with no search and no staging;
 * every other tile takes the staged path over the record's task range.
 *   tiles, num_tiles   device dc_tile[num_tiles]; num_tiles must equal the
 *                      planned count (else DC_ERR_SHAPE)
 * Other arguments as in dc_flush_bucket_buffers.  The plan is read on the
 * device and not checked: a stale plan can leave columns unwritten or give
 * wrong sums, but the kernel checks a whole tile's task before using its
 * pointers, so it never addresses memory outside the registered buffers. */
dc_status dc_flush_bucket_buffers_planned(int32_t W, int32_t dtype, int64_t bucket_numel,
                                          const dc_task* tasks, int32_t num_tasks,
                                          const void* const* in_ptrs, void* const* out_ptrs,
                                          const dc_comm* comms, int32_t num_comms, int32_t pre_div,
                                          const dc_tile* tiles, int64_t num_tiles, void* stream);

/* Host check of the tables of dc_flush_bucket_buffers (run once when the
 * buffers are registered): tasks sorted by offset, disjoint, numel >= 0,
 * inside [0, bucket_numel), comm in [0, num_comms); comms as in
 * dc_validate_tasks; a non-NULL input for every rank of every non-empty task;
 * no output overlapping another output or any input other than its own (an
 * output equal to its own input is the in-place case).  tasks, comms and the
 * two pointer tables are host copies (the pointer values are compared, never
 * dereferenced).  Returns DC_ERR_TASKS with a message naming the first
 * problem. */
dc_status dc_validate_buffer_tasks(int32_t W, int32_t dtype, const dc_task* tasks, int32_t num_tasks,
                                   int64_t bucket_numel, const dc_comm* comms, int32_t num_comms,
                                   const void* const* in_ptrs, void* const* out_ptrs);

/* Probe counts of one flush ([DS] "reduce_probe"), on the host from
 * metadata only (no device access, no synchronization).  tasks, owner (or
 * NULL for the empty map), pid_offsets/pids (the CSR of dc_partition_ids)
 * and comms are host arrays.  Holders of a param on a sub-communicator are,
 * in every block, the members whose in-block index is in its list. */
dc_status dc_probe_flush(int32_t W, int32_t dtype, const dc_task* tasks, int32_t num_tasks,
                         const int32_t* owner, int32_t num_params, const int32_t* pid_offsets,
                         const int32_t* pids, const dc_comm* comms, int32_t num_comms,
                         int32_t pre_div, dc_probe* out);

/* Holders of every task's param ([DS] problem statement: the copy-out after
 * the reduction writes each rank's gradient buffer and skips the ranks
 * whose buffer is empty; a rank keeps a buffer for a param when its
 * optimizer partition holds part of it, [DS] Design points).  Host only:
 * holders[t*W + r] = 1 when rank r's partition (its group rank, in every
 * block of a sub-communicator) is in the partition list of task t's param,
 * else 0 -- the ranks whose elements dc_probe_flush counts as kept, and the
 * outputs a fused flush (dc_flush_bucket_buffers) writes.
 *   tasks, num_tasks        host dc_task[num_tasks]; param in [0, num_params)
 *                           and comm in [0, num_comms) (else DC_ERR_TASKS)
 *   pid_offsets, pids       host CSR from dc_partition_ids
 *   comms, num_comms        host, as for dc_flush_bucket
 *   holders                 host uint8[num_tasks * W] out
 * A partition id outside its communicator is DC_ERR_TASKS. */
dc_status dc_holders(int32_t W, const dc_task* tasks, int32_t num_tasks, int32_t num_params,
                     const int32_t* pid_offsets, const int32_t* pids, const dc_comm* comms,
                     int32_t num_comms, uint8_t* holders);

/* Per-param ZeRO-2 partition sizes ([DS] "Follow-up": the ZeRO-2 owner path
 * sends every element to the rank whose partition holds it): for every
 * param of group g, param_part_size = part_size[g] (dc_partition_ids' S_g)
 * when g is on the data-parallel communicator -- the rule of
 * dc_build_owner_map: group_comm_size[g] == W and group rank i is global
 * rank i -- and 0 otherwise (such params keep AllReduce within their
 * blocks).  This is the part_size argument of dc_flush_bucket_zero2,
 * dc_plan_flush and dc_plan_relayout.
 *   group_begin, group_comm_size, group_rank_to_global  host, as for
 *                                                       dc_build_owner_map
 *   part_size          device int64[num_groups] from dc_partition_ids
 *   param_part_size    device int64[num_params] out */
dc_status dc_param_part_size(int32_t W, int32_t num_params, int32_t num_groups,
                             const int32_t* group_begin, const int32_t* group_comm_size,
                             const int32_t* group_rank_to_global, const int64_t* part_size,
                             int64_t* param_part_size, void* stream);

/* Relayout plan for a reduce-scatter over a bucket ([DS] "Describe
 * alternatives": a reduce-scatter needs the bucket laid out contiguously by
 * destination rank).  Every element of a task on the data-parallel comm whose
 * param has part_size > 0 belongs to partition
 * q = floor((flat_offset[param] + e) / part_size[param]); segment q of the
 * relaid bucket holds those elements in bucket order, and the segments follow
 * each other (q = 0..W-1).  Other tasks are not relaid.  Host only.
 *   tasks, num_tasks         host dc_task[] of the bucket (as validated by
 *                            dc_validate_tasks)
 *   flat_offset, part_size   host int64[num_params] (as for
 *                            dc_flush_bucket_zero2)
 *   pieces                   host dc_piece[pieces_capacity] out, sorted by
 *                            dst; NULL asks for the count only
 *   num_pieces               out: the number of pieces (at most num_tasks +
 *                            (W-1) per partitioned group in the bucket)
 *   seg_start                host int64[W+1] out: segment boundaries
 * Fewer than num_pieces slots is DC_ERR_SHAPE; a partition index outside
 * [0, W) is DC_ERR_TASKS. */
dc_status dc_plan_relayout(int32_t W, const dc_task* tasks, int32_t num_tasks,
                           const int64_t* flat_offset, const int64_t* part_size,
                           int32_t num_params, dc_piece* pieces, int32_t pieces_capacity,
                           int32_t* num_pieces, int64_t* seg_start);

/* Apply a relayout plan to every row: out[r][dst + i] = slab_in[r][bucket_col
 * + src + i] for each piece and i < len (pure data movement).
 *   slab_in, ld_in   device [W, ld_in]; the bucket is columns
 *                    [bucket_col, bucket_col + bucket_numel)
 *   out, ld_out      device [W, ld_out], ld_out >= out_numel; must not
 *                    overlap slab_in
 *   pieces           device dc_piece[num_pieces] sorted by dst
 * Only columns [0, out_numel) of `out` are written; a piece reaching outside
 * the bucket or outside [0, out_numel) is clipped, never followed. */
dc_status dc_relayout_bucket(int32_t W, int32_t dtype, const void* slab_in, int64_t ld_in,
                             void* out, int64_t ld_out, int64_t bucket_col, int64_t bucket_numel,
                             const dc_piece* pieces, int32_t num_pieces, int64_t out_numel,
                             void* stream);

/* Tile plan for dc_relayout_bucket_planned: the relayout above, taken to
 * the grain of the kernel's tiles once per bucket layout ([DS] Design
 * points: a bucket's layout is fixed, so what its flush needs is worked out
 * ahead of it).  The relaid bucket's columns [0, out_numel) fall into tiles
 * of 64 16-byte vectors (512 bf16 or 256 fp32 columns); one int64 per
 * tile, in an order private to the library, records where a tile copies
 * from when all of its columns belong to one piece (a column belongs to the
 * last piece whose dst is at or before it, if that piece reaches it) and
 * the piece's source run for the tile starts on a 16-byte vector of the
 * slab and stays in the bucket.  Host only.
 *   dtype, bucket_col, bucket_numel, pieces, num_pieces, out_numel
 *                    as for dc_relayout_bucket (pieces on the host, sorted
 *                    by dst as dc_plan_relayout writes them)
 *   tiles            host int64[tiles_capacity] out; NULL asks for the
 *                    count only
 *   num_tiles        out: ceil(ceil(out_numel / E) / 64), E = 8 (bf16) or
 *                    4 (fp32)
 * A negative piece length or pieces out of dst order is DC_ERR_ARG; fewer
 * than num_tiles slots is DC_ERR_SHAPE. */
dc_status dc_plan_relayout_tiles(int32_t dtype, int64_t bucket_col, int64_t bucket_numel,
                                 const dc_piece* pieces, int32_t num_pieces, int64_t out_numel,
                                 int64_t* tiles, int64_t tiles_capacity, int64_t* num_tiles);

/* dc_plan_relayout_tiles' records computed on the device, bit for bit, from
 * a piece table in device memory (one thread per destination tile, binary
 * search of the pieces' destinations): no host copy and no synchronization.
 *   pieces            device dc_piece[num_pieces]; must be sorted by dst with
 *                     no negative length (not checked here: another table
 *                     gives other records, every read and write stays in the
 *                     table and the plan)
 *   tiles, capacity   device int64[capacity] out; NULL asks for the count
 *                     only (nothing is launched)
 *   num_tiles         host out: the tile count (dc_plan_relayout_tiles')
 * Other arguments and checks as for dc_plan_relayout_tiles.  Stream-ordered. */
dc_status dc_plan_relayout_tiles_device(int32_t dtype, int64_t bucket_col, int64_t bucket_numel,
                                        const dc_piece* pieces, int32_t num_pieces,
                                        int64_t out_numel, int64_t* tiles, int64_t tiles_capacity,
                                        int64_t* num_tiles, void* stream);

/* dc_relayout_bucket from a tile plan: the same result, bit for bit.  A
 * tile with a record copies straight from it; any other tile searches the
 * pieces as dc_relayout_bucket does.  Arguments as for dc_relayout_bucket,
 * plus
 *   tiles, num_tiles  device int64[num_tiles] from dc_plan_relayout_tiles
 *                     on the same dtype, bucket, pieces and out_numel;
 *                     num_tiles must be the count it gives (else
 *                     DC_ERR_SHAPE)
 * A record is checked against the bucket before it is used: a plan made for
 * other pieces can misplace data inside the bucket's columns of `out`, but
 * never reads or writes outside them. */
dc_status dc_relayout_bucket_planned(int32_t W, int32_t dtype, const void* slab_in, int64_t ld_in,
                                     void* out, int64_t ld_out, int64_t bucket_col, int64_t bucket_numel,
                                     const dc_piece* pieces, int32_t num_pieces, int64_t out_numel,
                                     const int64_t* tiles, int64_t num_tiles, void* stream);

/* Reduce-scatter with variable shards: shard q is columns
 * [seg_start[q], seg_start[q+1]) of `in`, and
 *   out[q][k] = round_dtype(fold over r of pre(in[r][seg_start[q] + k]))
 * with the flush's fold and pre-division by W.
 *   seg_start     host int64[W+1], non-decreasing from 0, seg_start[W] <= ld_in
 *   out, ld_out   device [W, ld_out], ld_out >= the longest shard; no overlap */
dc_status dc_reduce_scatter_v(int32_t W, int32_t dtype, const void* in, int64_t ld_in, void* out,
                              int64_t ld_out, const int64_t* seg_start, int32_t pre_div,
                              void* stream);

/* ReduceScatter ([AG] duality with ReduceScatter: M elements in per node,
 * M/N out, a reduction plus a split).  With L = M / W:
 *   out[s][k] = round_dtype(fold over r of pre(in[r][s*L + k]))   k < L
 * using the flush's fold and pre-division (by W).
 *   in, ld_in     device [W, ld_in], ld_in >= M
 *   out, ld_out   device [W, ld_out], ld_out >= L; must not overlap `in`
 * M % W != 0 is DC_ERR_SHAPE (pad with zeros to a multiple of W). */
dc_status dc_reduce_scatter(int32_t W, int32_t dtype, const void* in, int64_t ld_in, void* out,
                            int64_t ld_out, int64_t M, int32_t pre_div, void* stream);

/* AllGather ([AG] semantic definition and Ring AllGather).  Shard s is
 * row s of `in` (L = shard_numel columns).
 *   DC_ORDER_RANK: out[i][s*L + k] = in[s][k] - every node ends with
 *                  [A_0, ..., A_{W-1}].
 *   DC_ORDER_RING: out[i][p*L + k] = in[(i - p) mod W][k] - position p of
 *                  node i holds the chunk a ring all-gather delivers at step
 *                  p (own chunk first, then one chunk per step from the left
 *                  neighbour).
 * step = -1 writes every position; step = s in [0, W) writes chunk s (rank
 * order) or position s (ring order) only, so a ring can be replayed step by
 * step.
 *   in, ld_in     device [W, ld_in], ld_in >= L
 *   out, ld_out   device [W, ld_out], ld_out >= W*L; must not overlap `in` */
dc_status dc_all_gather(int32_t W, int32_t dtype, const void* in, int64_t ld_in, void* out,
                        int64_t ld_out, int64_t shard_numel, int32_t order, int32_t step,
                        void* stream);

/* Ring-order ReduceScatter: the sum a ring reduce-scatter produces.  A ring
 * passes partial sums to the right, each node adding its own contribution,
 * so chunk s is folded in rank order s, s+1, ..., s-1 (mod W) instead of
 * 0..W-1 ([DS] Numerics: the summation order changes with the algorithm,
 * which is why owner and AllReduce results need not be bit-identical):
 *   out[s][k] = round_dtype(fold over j = 0..W-1 of pre(in[(s+j) mod W][s*L + k]))
 * Arguments, layout and checks as in dc_reduce_scatter. */
dc_status dc_reduce_scatter_ring(int32_t W, int32_t dtype, const void* in, int64_t ld_in,
                                 void* out, int64_t ld_out, int64_t M, int32_t pre_div,
                                 void* stream);

/* One step of an AllGather schedule ([AG] Ring AllGather, bidirectional
 * ring, Recursive Doubling AllGather) executed on one GPU: row i of `out`
 * ([W, W*L]) is node i's buffer, and every chunk is stored at its own index,
 * so after the last step every row is the rank-order concatenation.
 *   step 0            node i places its own shard: out[i][i*L + k] = in[i][k]
 *   DC_SCHED_RING     steps 1..W-1: node i receives chunk (i - step) mod W
 *                     from node i-1
 *   DC_SCHED_BIDIR    steps 1..ceil((W-1)/2): node i receives chunk
 *                     (i - step) mod W from node i-1 and chunk (i + step)
 *                     mod W from node i+1 (once when they coincide)
 *   DC_SCHED_RD       steps 1..log2 W (W a power of two): node i receives
 *                     the 2^(step-1) chunks held by node i XOR 2^(step-1)
 * Steps must run in order on the same buffers.  Other arguments as in
 * dc_all_gather; a step outside the schedule is DC_ERR_ARG. */
dc_status dc_all_gather_step(int32_t W, int32_t dtype, const void* in, int64_t ld_in, void* out,
                             int64_t ld_out, int64_t shard_numel, int32_t algo, int32_t step,
                             void* stream);

/* Replica-local accumulation ([MT] What: unreduced per-replica partial
 * sums accumulate locally across micro-batches).  fp32 only:
 *   acc[r][j] = acc[r][j] + x[r][j]        r < rows, j < M
 * and with init = 1 the accumulator starts from zero: acc = +0.0f + x.
 *   x, ld_x       device [rows, ld_x] fp32
 *   acc, ld_acc   device [rows, ld_acc] fp32, updated in place; may equal x */
dc_status dc_accumulate(int32_t rows, const float* x, int64_t ld_x, float* acc, int64_t ld_acc,
                        int64_t M, int32_t init, void* stream);

/* Deferred cross-replica reduce ([MT] What: the single all-reduce that
 * update() emits).  fp32 only:
 *   out[i][j] = fold over r = 0..W-1 of acc[r][j]        i < out_rows, j < M
 * out_rows is 1 (one reduced copy) or W (every replica gets the sum).  With
 * out_rows = 1 and W rows of one micro-batch this is also the
 * per-micro-batch reduce of the status quo.
 *   acc, ld_acc   device [W, ld_acc] fp32
 *   out, ld_out   device [out_rows, ld_out] fp32; may equal acc (same ld) */
dc_status dc_deferred_reduce(int32_t W, const float* acc, int64_t ld_acc, float* out,
                             int64_t ld_out, int64_t M, int32_t out_rows, void* stream);

/* Accumulation and the deferred reduce fused for the last micro-batch of a step: the same fp32
 * operations as dc_accumulate followed by dc_deferred_reduce, in one pass
 * (bit-identical results), without writing the accumulator and reading it
 * back ([MT] What: the accumulated partial sums feed the single reduce in
 * update()).  For every j < M:
 *   a_r = init ? +0.0f + x[r][j] : acc[r][j] + x[r][j]      r < W
 *   acc[r][j] = a_r                      only when keep_acc = 1
 *   out[i][j] = fold over r = 0..W-1 of a_r                  i < out_rows
 *   x, ld_x       device [W, ld_x] fp32
 *   acc, ld_acc   device [W, ld_acc] fp32 (not read when init = 1); may
 *                 equal x (same ld)
 *   out, ld_out   device [out_rows, ld_out] fp32, out_rows 1 or W; may equal
 *                 acc (same ld) only when keep_acc = 0; must not overlap x
 * Algorithmic bytes: W*M*4 read of x, W*M*4 read of acc unless init,
 * W*M*4 written to acc if keep_acc, out_rows*M*4 written. */
dc_status dc_accumulate_reduce(int32_t W, const float* x, int64_t ld_x, float* acc, int64_t ld_acc,
                               int32_t init, int32_t keep_acc, float* out, int64_t ld_out,
                               int32_t out_rows, int64_t M, void* stream);

/* fp32 -> bf16 with the rounding the flush uses (round to nearest even, NaN
 * -> 0x7FC0|sign), n elements, device arrays; a self-check of the
 * conversion on the GPU. */
dc_status dc_round_bf16(const float* in, uint16_t* out, int64_t n, void* stream);

/* Plain 16-byte streaming copy of `bytes` (a multiple of 16; both pointers
 * 16-byte aligned, not overlapping): the achievable-bandwidth reference the
 * measurements compare against. */
dc_status dc_stream_copy(const void* src, void* dst, int64_t bytes, void* stream);

/* Access-mix reference for measurements: for each of `nvec` 16-byte column
 * vectors, read it from rows_read rows of `src` (rows src_ld_vec vectors
 * apart), xor them, and store the result to rows_written rows of `dst`
 * (rows dst_ld_vec vectors apart).  No other arithmetic, so its bandwidth is
 * what the memory system gives the flush's access mix (W rows read, one row
 * or W rows written).  rows_read is 4, 8 or 16 and rows_written 1 or
 * rows_read (else DC_ERR_UNSUPPORTED); pointers 16-byte aligned; the two
 * regions must not overlap. */
dc_status dc_stream_rows(const void* src, int64_t src_ld_vec, int32_t rows_read, void* dst,
                         int64_t dst_ld_vec, int32_t rows_written, int64_t nvec, void* stream);

/* The access-mix reference at a launch shape of the planned flush: the same
 * xor stream as dc_stream_rows, but each one-wave workgroup takes `group`
 * (1, 2 or 4) runs of 64 vectors -- with one row written their results are
 * stored together after the last load -- at most `cap` workgroups stay
 * resident per compute unit (0: no cap, at most 64), and the stores use the
 * planned flush's cache policies.  A sweep over shapes that includes a
 * kernel's own gives a reference its access mix cannot beat with xor for
 * arithmetic.  Other arguments and checks as in dc_stream_rows, except
 * that rows_read 1 with rows_written 4, 8 or 16 (the all-gather's mix: one
 * row read, every row written) and rows_read 8 with rows_written 4 (the
 * W = 4 fused accumulate-reduce's: accumulators and micro-batch read, every
 * replica row written) are also supported; a group outside {1, 2, 4} is
 * DC_ERR_UNSUPPORTED. */
dc_status dc_stream_rows_shaped(const void* src, int64_t src_ld_vec, int32_t rows_read, void* dst,
                                int64_t dst_ld_vec, int32_t rows_written, int64_t nvec,
                                int32_t group, int32_t cap, void* stream);

/* ---- A layer's products and the owner's update --------------------------
 *
 * These take matrices where a model keeps them: element-aligned bases (else
 * DC_ERR_ALIGN) and any row stride of at least the row's length, in
 * elements.  16-byte aligned operands with strides of whole 16 bytes run
 * faster.  What an output's row holds between its length and its stride stays
 * as it was.  Outputs must not overlap inputs or other outputs (DC_ERR_ARG)
 * except where said; two matrices that interleave as column ranges of rows
 * with one common stride do not overlap, nor does a single row that lies between
 * another matrix's rows.  Sizes are at most 2^28 and the
 * elements of one matrix at most 2^36 (2^20 and 2^34 for dc_matrix), else
 * DC_ERR_SHAPE.
 * A workspace is device memory, 16-byte aligned, of at least the bytes that
 * the query gives for the same arguments (else DC_ERR_SHAPE; NULL is allowed
 * when it gives 0); it is scratch: it need not be cleared, holds nothing
 * between calls, and must not be shared by calls that may run at once. */

/* Bytes of workspace of dc_linear, dc_linear_backward and
 * dc_bias_act_backward for these sizes.  Host only. */
dc_status dc_linear_workspace(int32_t dtype, int64_t T, int64_t N, int64_t K, int64_t* bytes);
dc_status dc_linear_backward_workspace(int32_t dtype, int64_t T, int64_t N, int64_t K, int64_t* bytes);
dc_status dc_bias_act_workspace(int32_t dtype, int64_t T, int64_t N, int64_t* bytes);

/* The kernel that a product runs on, as the library chooses it from types and
 * sizes: out[0] its square tile (256, 128 or 64; 0: the kernel for up to 64
 * rows), out[1] the stages of its loads (where operands and strides are whole
 * 16 bytes; others go through registers), out[2] the parts that its sum is cut
 * into.  For profiles and tests; nothing depends on it.  Host only.
 *   product   DC_PRODUCT_FORWARD (dc_linear), DC_PRODUCT_DX or DC_PRODUCT_DW
 *             (dc_linear_backward)
 *   out       host int32[3] */
dc_status dc_linear_form(int32_t dtype, int32_t product, int64_t T, int64_t N, int64_t K, int32_t* out);

/* Linear layer on T rows (tokens), N outputs, K inputs:
 *   pre[t][n] = sum_k x[t][k] w[n][k] + bias[n]
 *   y[t][n]   = act(pre[t][n]) + residual[t][n]
 * Sums, activation and residual in fp32, y and pre each rounded once.
 *   x, ld_x          device [T, ld_x], ld_x >= K
 *   w, ld_w          device [N, ld_w], ld_w >= K
 *   bias             device [N] or NULL
 *   residual, ld_res device [T, ld_res] or NULL; may be y itself (same ld)
 *   act              DC_ACT_*
 *   pre, ld_pre      device [T, ld_pre] out or NULL: what
 *                    dc_bias_act_backward reads
 *   y, ld_y          device [T, ld_y] out
 * T = 0 writes nothing; N and K are at least 1. */
dc_status dc_linear(int32_t dtype, int64_t T, int64_t N, int64_t K, const void* x, int64_t ld_x,
                    const void* w, int64_t ld_w, const void* bias, const void* residual,
                    int64_t ld_res, int32_t act, void* pre, int64_t ld_pre, void* y, int64_t ld_y,
                    void* workspace, int64_t workspace_bytes, void* stream);

/* Backward of the bias and the activation:
 *   dz[t][n] = dy[t][n] act'(pre[t][n])         rounded once
 *   db[n]    = (accumulate ? db[n] : 0) + sum_t dy[t][n] act'(pre[t][n])
 * the sum in fp32 over the unrounded products, in an order fixed by the
 * sizes.  The residual's gradient is dy itself.  act'(0) of relu is 0.
 *   dy, ld_dy    device [T, ld_dy]
 *   pre, ld_pre  device [T, ld_pre]; NULL with DC_ACT_NONE (else DC_ERR_NULL)
 *   dz, ld_dz    device [T, ld_dz] out, or NULL; may be dy itself (same ld)
 *   grad_dtype   of db: DC_F32, or dtype
 *   db           device [N], or NULL
 * T = 0 gives db's empty sum. */
dc_status dc_bias_act_backward(int32_t dtype, int64_t T, int64_t N, const void* dy, int64_t ld_dy,
                               const void* pre, int64_t ld_pre, int32_t act, void* dz,
                               int64_t ld_dz, int32_t grad_dtype, void* db, int32_t accumulate,
                               void* workspace, int64_t workspace_bytes, void* stream);

/* Backward of the products:
 *   dx[t][k] = sum_n dz[t][n] w[n][k]                              (dtype)
 *   dw[n][k] = (accumulate ? dw[n][k] : 0) + sum_t dz[t][n] x[t][k] (grad_dtype)
 * in fp32, rounded once.  With accumulate and DC_F32, dw is a parameter's
 * place in a replica's accumulator row ([MT] What: micro-batch gradients add
 * up locally), with no gradient written and read in between.
 *   dz, ld_dz   device [T, ld_dz], ld_dz >= N
 *   w, ld_w     device [N, ld_w]; read only when dx is given
 *   x, ld_x     device [T, ld_x]; read only when dw is given
 *   dx, ld_dx   device [T, ld_dx] out, or NULL
 *   grad_dtype  of dw: DC_F32, or dtype
 *   dw, ld_dw   device [N, ld_dw], or NULL
 * T = 0 gives dw's empty sum. */
dc_status dc_linear_backward(int32_t dtype, int64_t T, int64_t N, int64_t K, const void* dz,
                             int64_t ld_dz, const void* w, int64_t ld_w, const void* x, int64_t ld_x,
                             void* dx, int64_t ld_dx, int32_t grad_dtype, void* dw, int64_t ld_dw,
                             int32_t accumulate, void* workspace, int64_t workspace_bytes,
                             void* stream);

/* Bytes of workspace of dc_orthogonalize (out_dtype = dtype) and
 * dc_muon_update (out_dtype = weight_dtype) for this list (its rows and
 * cols): at most 4 GiB and 256 KiB, or what its largest matrix needs, as
 * longer lists are worked off in parts.  Host only. */
dc_status dc_orthogonalize_workspace(int32_t dtype, int32_t out_dtype, int32_t hold,
                                     const dc_matrix* mats, int32_t num, int64_t* bytes);

/* The same for the products of matrix `index` of a list: out[3 k ..] for A (k =
 * 0), B (1), a step's X (2) and the last step's (3).
 *   update  1: dc_muon_update, 0: dc_orthogonalize
 *   out     host int32[12] */
dc_status dc_orthogonalize_form(int32_t dtype, int32_t out_dtype, int32_t hold, const dc_matrix* mats,
                                int32_t num, int32_t update, int32_t index, int32_t* out);

/* Every matrix orthogonalised by Newton-Schulz products.  With X the
 * gradient (its transpose where rows > cols):
 *   X <- X / (|X|_F + eps)
 *   for every step (a, b, c):  A = X XT,  X <- a X + (b A + c A A) X
 * and X (transposed back) is written to out: the singular vectors stay, the
 * singular values go through the odd polynomials a s + b s^3 + c s^5.
 * X, A and B are held in fp16, by powers of two that the polynomials' bounds
 * keep from overflowing, with fp32 sums: a pair of them (22 bits), which leaves
 * about 1e-6 of |out|_F (up to 2e-6; the same steps in fp32 leave 0.3e-6 to
 * 3.6e-6), or one (11 bits), which leaves about 1.5e-3 on matrices of 256 and more a side, up
 * to 1e-2 on small ones, and takes a third of the products.  hold DC_HOLD_AUTO takes pairs where the gradients or the
 * output are fp32 or the smaller side is under 256, else one; DC_HOLD_ONE and
 * DC_HOLD_PAIR are the caller's choice for the whole list.  |X|_F is summed in
 * fp64.  A zero matrix gives zero (NaN when eps is 0); a NaN or
 * infinity anywhere gives NaN in the whole of its matrix and no other.
 *   mats, num       host dc_matrix[num], num <= 2^20; out has the dtype of the gradients
 *                   and may be the gradient itself (same ld), otherwise
 *                   overlaps no gradient and no other out
 *   steps, coeffs   host float[steps][3], 1 <= steps <= DC_NS_MAX_STEPS; the
 *                   bound on the singular values must stay under 64
 *                   (else DC_ERR_ARG: the steps diverge)
 *   eps             >= 0 */
dc_status dc_orthogonalize(int32_t dtype, int32_t hold, const dc_matrix* mats, int32_t num,
                           int32_t steps, const float* coeffs, float eps, void* workspace,
                           int64_t workspace_bytes, void* stream);

/* The owner's update of whole matrices from their reduced gradients ([DS]
 * problem statement: after reduce-to-owner one rank holds a parameter's whole
 * gradient).  For every matrix:
 *   m <- mu m + g                              (fp32, stored)
 *   u  = nesterov ? mu m + g : m
 *   O  = u orthogonalised, as dc_orthogonalize (held as hold says)
 *   w <- (1 - l weight_decay) w - l s O        (fp32, rounded to weight_dtype)
 * with l = lr, times *lr_scale when given (device float[1], read when the
 * work runs: a recorded graph follows a schedule through it), and s the
 * shape's factor (DC_SCALE_*).
 *   dtype         of the gradients; weight_dtype: of out, the weights
 *   mats, num     host dc_matrix[num]; weights and momenta overlap nothing
 * Other arguments as in dc_orthogonalize. */
dc_status dc_muon_update(int32_t dtype, int32_t weight_dtype, int32_t hold,
                         const dc_matrix* mats, int32_t num, float lr, const float* lr_scale,
                         float mu, int32_t nesterov, float weight_decay, int32_t scale_mode,
                         int32_t steps, const float* coeffs, float eps, void* workspace, int64_t workspace_bytes,
                         void* stream);

/* ---- Clipping by the global norm -----------------------------------------
 *
 * Between the reduction and the update: over a list of gradients of both
 * dtypes, as the flush or the deferred reduce left them, the global norm
 *   n = sqrt(sum over the counted rows of every gradient of g^2)
 * and
 *   c = n + eps <= max_norm ? 1 : max_norm / (n + eps),   out = c g
 * over all rows.  Squares and sums are fp64, in an order fixed by the list's sizes and
 * strides; c is rounded once to fp32 (under 2^-126 to the bits that are left
 * there), c g to fp32 and then to the dtype.  An infinity among the counted
 * gradients gives c = 0 (and NaN where it stands), a NaN gives NaN throughout:
 * read *norm to pass such a step over.  Rules of the section above hold, with
 * 2^36 elements per gradient and 2^44 per row stride. */

/* Bytes of workspace of dc_grad_norm and dc_grad_clip.  Host only. */
dc_status dc_grad_clip_workspace(int64_t* bytes);

/* The norm alone.
 *   grads, num   host dc_gradient[num], num <= 2^20; out is not read
 *   accumulate   1: *squares is added to, so that lists, or ranks that add
 *                their *squares up, share one norm (squares is then required)
 *   squares      device double[1] out, the sum of squares; or NULL
 *   norm         device float[1] out, sqrt(*squares); or NULL */
dc_status dc_grad_norm(const dc_gradient* grads, int32_t num, int32_t accumulate, double* squares,
                       float* norm, void* workspace, int64_t workspace_bytes, void* stream);

/* Clipping.  No out overlaps another gradient's grad or out; with `squares`,
 * norm and coef, none overlaps anything else.
 *   squares      device double[1], the sum of squares to clip by (not
 *                changed), or NULL: that of this list
 *   max_norm     >= 0, may be infinite (c = 1); eps >= 0, finite
 *   norm, coef   device float[1] out: n and c; or NULL
 * Gradients clipped in place by a factor of 1 are not touched. */
dc_status dc_grad_clip(const dc_gradient* grads, int32_t num, const double* squares, float max_norm,
                       float eps, float* norm, float* coef, void* workspace, int64_t workspace_bytes,
                       void* stream);

/* ---- The embedding ---------------------------------------------------------
 *
 * Rules of the layer's products hold; T at most 2^26, D at most 2^22. */

/* Lookup of T tokens in a table of `rows` rows and D columns, with scaling:
 *   out[t] = scale E[ids[t]]          in fp32, rounded once
 * An id outside [0, rows) gives zeros: padding, or a token of another rank's
 * part of the table.
 *   id_bytes         4 or 8 (else DC_ERR_DTYPE): signed ids of 32 or 64 bits
 *   ids              device [T], aligned to their size
 *   table, ld_table  device [rows, ld_table]
 *   out, ld_out      device [T, ld_out] out */
dc_status dc_embedding(int32_t dtype, int32_t id_bytes, int64_t T, int64_t rows, int64_t D, const void* ids,
                       const void* table, int64_t ld_table, float scale, void* out, int64_t ld_out,
                       void* stream);

/* Bytes of workspace of dc_embedding_backward.  Host only. */
dc_status dc_embedding_backward_workspace(int32_t dtype, int64_t T, int64_t rows, int64_t D,
                                          int64_t* bytes);

/* The table's gradient:
 *   dE[v] = (accumulate ? dE[v] : 0) + scale sum over {t: ids[t] = v} of dy[t]
 * in fp32, every row's sum in the order of its tokens (in parts of up to 32
 * tokens fixed by the ids, added in order in fp64), rounded once.  With accumulate, rows that no id names are neither
 * read nor written; without it they become zeros.  An id outside [0, rows)
 * gives nothing.  With accumulate and DC_F32, dE is a parameter's place in a
 * replica's accumulator row ([MT] What: micro-batch gradients add up locally).
 *   dy, ld_dy    device [T, ld_dy], ld_dy >= D; a row of a dropped id is not read
 *   grad_dtype   of dtable: DC_F32, or dtype
 *   dtable, ld   device [rows, ld], ld >= D */
dc_status dc_embedding_backward(int32_t dtype, int32_t id_bytes, int64_t T, int64_t rows, int64_t D,
                                const void* dy, int64_t ld_dy, const void* ids, float scale,
                                int32_t grad_dtype, void* dtable, int64_t ld, int32_t accumulate,
                                void* workspace, int64_t workspace_bytes, void* stream);

/* ---- Norms around a block ---------------------------------------------------
 *
 * Rules of the layer's products hold; D is at most 16384, the columns that a
 * workgroup holds in registers (else DC_ERR_UNSUPPORTED). */

/* The norm after a block, its gate and the residual's scale, and the norm
 * before the next block, on T rows (tokens) of D columns:
 *   u[t] = (offset + post_gain) h[t] / sqrt(mean(h[t]^2) + eps)
 *   s[t] = x[t] + scale gate[t / (T / gate_rows)] u[t]
 *   y[t] = (offset + gain) s[t] / sqrt(mean(s[t]^2) + eps)
 * in fp32 with the means' sums in fp64, s and y each rounded once (y from the
 * s before its rounding); with eps = 0 rows of subnormal values are normed like
 * others, and a row of zeros gives NaN.  What is NULL falls away: without post_gain u = h, without gate it is 1,
 * without h s = x, without gain there is no y; h or gain is needed, and h for
 * post_gain and gate.
 *   x, ld_x          device [T, ld_x]: the residual stream
 *   h, ld_h          device [T, ld_h] or NULL: the block's output
 *   post_gain, gain  device [D] or NULL
 *   gate, ld_gate    device [gate_rows, ld_gate] or NULL; gate_rows >= 1 divides
 *                    T, and every row serves T / gate_rows tokens in turn
 *   s, ld_s          device [T, ld_s] out, or NULL; with h only; may be x (same
 *                    ld) or h
 *   y, ld_y          device [T, ld_y] out; with gain only; may be x or h,
 *                    where s is not
 * T = 0 writes nothing (and asks for no pointer). */
dc_status dc_norm(int32_t dtype, int64_t T, int64_t D, const void* x, int64_t ld_x, const void* h,
                  int64_t ld_h, const void* post_gain, const void* gate, int64_t gate_rows,
                  int64_t ld_gate, const void* gain, float scale, float offset, float eps, void* s,
                  int64_t ld_s, void* y, int64_t ld_y, void* stream);

/* Bytes of workspace of dc_norm_backward.  Host only. */
dc_status dc_norm_backward_workspace(int32_t dtype, int64_t T, int64_t D, int64_t gate_rows,
                                     int64_t* bytes);

/* Its backward.  With n = s / sqrt(mean(s^2) + eps), m = h / sqrt(mean(h^2) + eps)
 * (h without post_gain), r2 and r1 those factors:
 *   q = (offset + gain) dy,  dx = ds + r2 (q - n mean(q n))
 *   dgain (+)= sum_t dy n
 *   v = scale gate dx,  dgate (+)= sum over the row's tokens of scale dx u
 *   g = (offset + post_gain) v,  dh = r1 (g - m mean(g m))  (v without post_gain)
 *   dpost_gain (+)= sum_t v m
 * in fp32 with the means' sums in fp64, from s as it is stored; sums over
 * tokens are fp32 in an order fixed by the sizes (the parts that a gate row's
 * sum may come in are added in fp64); each output is rounded once,
 * dx and dh from the same unrounded dx.
 *   dy, ld_dy        device [T, ld_dy]: y's gradient; read with gain
 *   ds, ld_ds        device [T, ld_ds] or NULL (0): what reaches s from later
 *   s, ld_s          device [T, ld_s]: read with gain
 *   dx, ld_dx        device [T, ld_dx] out, or NULL; may be ds, dy, s or h
 *   dh, ld_dh        device [T, ld_dh] out, or NULL; with h only; may be ds,
 *                    dy, s or h, where dx is not
 *   grad_dtype       of dgain, dpost_gain and dgate: DC_F32, or dtype
 *   dgain, dpost_gain  device [D], or NULL
 *   dgate, ld_dgate  device [gate_rows, ld_dgate], or NULL
 *   accumulate       1: added to what dgain, dpost_gain and dgate hold
 * Other arguments as for dc_norm.  T = 0 gives the gradients' empty sums. */
dc_status dc_norm_backward(int32_t dtype, int64_t T, int64_t D, const void* dy, int64_t ld_dy,
                           const void* ds, int64_t ld_ds, const void* s, int64_t ld_s, const void* h,
                           int64_t ld_h, const void* post_gain, const void* gate, int64_t gate_rows,
                           int64_t ld_gate, const void* gain, float scale, float offset, float eps,
                           void* dx, int64_t ld_dx, void* dh, int64_t ld_dh, int32_t grad_dtype,
                           void* dgain, void* dpost_gain, void* dgate, int64_t ld_dgate,
                           int32_t accumulate, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DC_H */
