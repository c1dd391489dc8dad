/*
 * kvl.h -- layer-wise paged KV block reshuffle on one GPU (GB300, sm_103a).
 *
 * C ABI of libkvl.so.  Every buffer is caller memory; the library allocates nothing,
 * keeps no per-call state and never synchronises the caller's stream except in
 * kvl_read_status.  All calls only ENQUEUE work on `stream` (a cudaStream_t passed as
 * void*, NULL = the legacy default stream): results are valid once the caller has
 * synchronised that stream or an event recorded after the call (DualPath KV Loading,
 * "Dual-Path Loading", pe_read_path listing: every write is followed by a wait for
 * its completion before the buffer is used).
 *
 * What the calls compute (the pages' objects, per layer l):
 *   hit_full_block       persisted cross-layer KV of the hit prefix, semantic view
 *                        [T_hit, L, C_KV]; here [T_hit, L, P, Rp] bytes, token-major
 *                        (DualPath KV Loading, "Dual-Path Loading", objects table)
 *   hit_layer[l]         = hit_full_block[:, l], [T_hit, P, Rp]          (slice_layer)
 *   miss_layer[l]        freshly computed KV of the appended tokens, [T_miss, P, Rp]
 *   complete_layer[l]    hit rows then miss rows, [T_all, P, Rp]   (concatenate_tokens)
 *   paged pool           blocks of [B_tokens, H, d] linked per sequence by a block
 *                        table (Tutti 阅读笔记, 前置知识 3 "分页 KV 内存管理", eq. (2))
 *   K / V objects        one K and one V object per (layer, block): 2*L*ceil(T/B)
 *                        objects per sequence (Tutti 阅读笔记, 前置知识 5, eqs. (3)(4);
 *                        设计一 §3.1: one GPU file per block holding 2L objects)
 *
 * Geometry symbols: L layers, P planes per token (2 = K and V for head-split KV,
 * 1 = one latent vector), B tokens per block, Rp bytes per token per plane
 * (H_kv*d*2 for bf16 heads, C_KV*2 for a bf16 latent vector), R = P*Rp, N pool blocks.
 * T_all = T_hit + T_miss, nblk = ceil(T_all / B), nsrc = ceil(T_hit / B).
 *
 * Layouts (byte addresses; every one is a plain byte copy, values never pass through
 * arithmetic, so the results are bit-exact):
 *   hit token t (t < T_hit), layer l, plane p:
 *       hit_src + sb(t/B)*hit_block_stride + (t%B)*hit_token_stride
 *               + l*hit_layer_stride + p*Rp,   sb(j) = hit_src_table ? hit_src_table[j] : j
 *       (a contiguous full block [T_hit, L, P, Rp] has block stride B*L*R, token
 *        stride L*R, layer stride R; a "Full Block" store of [B, L, P, Rp] blocks at
 *        shuffled places uses hit_src_table)
 *   miss token t (T_hit <= t < T_all):
 *       miss_src + (t - T_hit)*miss_token_stride + l*miss_layer_stride + p*Rp
 *   pool, block b, slot s:  pool + (((l*P + p)*N + b)*B + s)*Rp   ([L][P][N][B][Rp])
 *   object (l, p, j) of a request, B*Rp bytes:
 *       objects + l*obj_layer_stride + p*obj_plane_stride + j*obj_block_stride
 *       layer-major [L][P][nblk][B][Rp] (object id (l*P + p)*nblk + j): strides
 *         (P*nblk*B*Rp, nblk*B*Rp, B*Rp);
 *       block-major [nblk][L][P][B][Rp], one "GPU file" per block holding its 2L
 *         objects (Tutti 阅读笔记, 设计一 §3.1 and 伪代码 1: file offset = file id x
 *         file stride + layer x per-layer size): strides (P*B*Rp, B*Rp, L*P*B*Rp)
 *   hit_out / complete_out: request r's token t at row hit_off[r] + t / tok_off[r] + t
 *       of R bytes ([sum T_hit][P][Rp] / [sum T_all][P][Rp], requests in order)
 *   block tables: one int32 array, request r's nblk entries at blk_off[r] (requests
 *       packed back to back in order); one table serves every layer and plane.
 *
 * Partial blocks: the scatter writes only slots t < T_all; later slots of the last
 * block keep their bytes.  Objects always carry whole blocks (fixed object size
 * B*Rp), so a partial block's object carries whatever those slots hold.
 *
 * Alignment: Rp, every stride and every buffer address must be multiples of 16 bytes.
 * Size: Rp, and R for kvl_slice_layer, at most 32 KiB (one shared-memory stage).
 * Aliasing: sources, pool, objects and outputs must not overlap (undefined otherwise);
 * with an injective block table every destination byte has exactly one writer.
 *
 * A plan records the request array and block tables it was built from; a call that
 * passes other arrays with that plan is refused on the device (KVL_EINVAL).
 *
 * Errors: problems the host can see (null or misaligned arguments, a bad geometry,
 * a layer outside [0, L), a plan too small) are returned at once and nothing is
 * launched.  Problems only the device can see (negative counts, misaligned request
 * fields, block ids out of range, duplicate block ids) are recorded in the plan's
 * status word: the offending work is skipped, nothing traps, and every later call
 * made with that plan does nothing until the plan is rebuilt.  Of the call that meets
 * the problem, any part of its other work may be left undone (its CTAs stop once they
 * see the status).  kvl_read_status reads the word back.  KVL_ECUDA reports a failed
 * launch.
 */
#ifndef KVL_H
#define KVL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t kvl_status;

#define KVL_OK 0
#define KVL_EINVAL 1 /* bad argument or geometry, negative count, null pointer */
#define KVL_EALIGN 2 /* pointer, stride or Rp not a multiple of 16 bytes */
#define KVL_ERANGE 3 /* block id outside the pool / source, or plan capacity exceeded */
#define KVL_EDUP 4   /* a pool block id used twice (only with check_injective) */
#define KVL_ECUDA 5  /* a CUDA launch or copy failed */
#define KVL_ETIMEOUT 6 /* a copy kernel's bounded wait on its own copies ran out (detail = CTA) */

#define KVL_GATHER 0      /* kvl_gather_layer_objects: pool -> objects */
#define KVL_SCATTER_BACK 1 /* kvl_gather_layer_objects: objects -> pool */

/* Geometry shared by every request of a batch (host memory). */
typedef struct kvl_geom {
    int32_t n_layers;        /* L */
    int32_t n_planes;        /* P: 2 = K,V planes; 1 = latent vector */
    int32_t block_tokens;    /* B: tokens per paged block */
    int32_t plane_row_bytes; /* Rp: bytes per token per plane, multiple of 16 */
    int64_t pool_blocks;     /* N: physical blocks in the pool */
} kvl_geom;

/* Launch options of a copy call (host memory; NULL = defaults). */
typedef struct kvl_launch {
    int32_t max_ctas; /* 0: one CTA on every SM (the whole GPU); k > 0: at most k CTAs,
                         i.e. the copy occupies at most k SMs and leaves the rest to
                         concurrent work (an I/O SM budget, as Tutti 阅读笔记 设计二
                         gives its I/O kernels a fixed SM partition) */
    int32_t flags;    /* 0, or KVL_LAUNCH_HOST_SRC or KVL_LAUNCH_HOST_DST (not both),
                         optionally OR KVL_LAUNCH_OVERLAP_PREVIOUS, KVL_LAUNCH_SHARE_SMS
                         and / or KVL_LAUNCH_PLAN_READY */
} kvl_launch;

/* The copy's sources (resp. destinations) are pinned host memory mapped into the
 * device address space (cudaHostAlloc / cudaHostRegister): e.g. DualPath's host
 * buffers, the full prompt KV held in Grace memory (DualPath KV Loading, "Dual-Path
 * Loading": pe_buffer / de_buffer and the final H2D into the HBM cache).  That side
 * is read (written) with ordinary 16-byte SM loads (stores) over NVLink-C2C; the HBM
 * side keeps the bulk-copy path.  Without the flag every buffer must be device memory. */
#define KVL_LAUNCH_HOST_SRC 1
#define KVL_LAUNCH_HOST_DST 2

/* The call may start copying before the kernel enqueued just before it on the stream
 * has finished, on the SMs that kernel has already left; it still finishes only after
 * that kernel has (so a later call without the flag sees both complete).  Meant for
 * the layer-wise pipeline's consecutive launches of one op on successive layers
 * (Tutti 阅读笔记, 伪代码 1: one I/O launch per layer; layers touch disjoint pool
 * regions), so that one launch's ramp-up fills the previous launch's tail.
 * The caller guarantees that the call touches no byte that the kernels it may overlap
 * write, and writes no byte that they read: the kernel just before it and, when that
 * call carried the flag too, the kernels that call may overlap in turn.  Reads of the
 * same plan, requests and tables are fine, but the plan's own kernels write the plan:
 * the first copy call after kvl_batch_plan must not carry the flag.  A call for the same plan, layer and op as
 * the kernel before it must not carry the flag (the two would share a work counter).
 * A call that overlaps a failing one may still copy: the failure shows in the plan's
 * status (kvl_read_status) once both have finished. */
#define KVL_LAUNCH_OVERLAP_PREVIOUS 4

/* Performance hint: the call's CTAs take half of an SM's shared memory (a 96 KiB
 * pipeline instead of 192 KiB), so that a CTA of the next launch, if that one carries
 * KVL_LAUNCH_OVERLAP_PREVIOUS, can run beside it on the same SM.  Set it on the call
 * just before a run of overlapping calls; KVL_LAUNCH_OVERLAP_PREVIOUS implies it.  A
 * call that runs alone is faster without it.  The host-memory variants ignore it. */
#define KVL_LAUNCH_SHARE_SMS 8

/* The caller declares that the plan (and the request array and tables it was built
 * from) was complete before the kernel enqueued just before this call began: no
 * kernel that may still run writes it, other than the copy calls' own claim counters
 * and status word.  True of every copy call of a layer-wise pipeline except the first
 * one after kvl_batch_plan.  A call that must wait for the kernel before it (no
 * KVL_LAUNCH_OVERLAP_PREVIOUS) then checks the plan, reads and decodes its first work
 * items and prefetches their source rows into L2 (cp.async.bulk.prefetch) while that
 * kernel drains, and waits only before its first copy; L2 is the device's point of
 * coherence, so rows the previous kernel writes are still read as it leaves them.
 * Results are the same with or without the flag; with a plan that is not complete,
 * undefined.  Ignored with KVL_LAUNCH_OVERLAP_PREVIOUS and by the host-memory
 * variants. */
#define KVL_LAUNCH_PLAN_READY 16

/* One request (device memory: the calls take an array of these in device memory).
 * All strides are in bytes. */
typedef struct kvl_request {
    const void *hit_src;          /* full block of the hit prefix (NULL if t_hit == 0) */
    const int32_t *hit_src_table; /* NULL, or nsrc full-block ids (device memory) */
    int64_t hit_src_blocks;       /* full blocks present at hit_src (bounds the ids) */
    int64_t hit_block_stride;
    int64_t hit_token_stride;
    int64_t hit_layer_stride;
    const void *miss_src;         /* miss KV (NULL if t_miss == 0) */
    int64_t miss_token_stride;
    int64_t miss_layer_stride;
    void *objects;                /* this request's K/V objects (NULL if never gathered) */
    int64_t obj_layer_stride;
    int64_t obj_plane_stride;
    int64_t obj_block_stride;
    int32_t t_hit;
    int32_t t_miss;
} kvl_request;

/* Bytes of device memory a plan for n_req requests in this geometry needs (0 for a
 * bad geometry).  The plan holds at most pool_blocks work items (injective tables
 * never need more), a 128-byte record per item and a claim counter per (layer, op). */
size_t kvl_plan_bytes(const kvl_geom *geom, int32_t n_req);

/* Plan layout, for callers that read the plan's arrays (byte offsets into the plan):
 * off[0] header, off[1] tok_off (int64[n_req+1]), off[2] hit_off (int64[n_req+1]),
 * off[3] blk_off (int64[n_req+1]), off[4] item_req (int32[pool_blocks]),
 * off[5] item_blk (int32[pool_blocks]), off[6] item records (always at byte 256),
 * off[7] claim counters, off[8] injectivity bitmap (the last section), off[9] total
 * bytes, off[10] tensor maps (6 x 128 bytes per request, starting at the first
 * 128-byte boundary at or after the plan's address + off[10], then an int32 of map
 * flags per request).  Sections are not
 * placed in index order.  The header's first int32 is the status and its int64 at
 * byte 16 the item count. */
void kvl_plan_layout(const kvl_geom *geom, int32_t n_req, size_t off[11]);

/* kvl_batch_plan -- the batch's work list, built on the device.
 * Computes exclusive prefix sums over requests of T_all (tok_off), T_hit (hit_off)
 * and nblk (blk_off), and the work list item i = blk_off[r] + j -> (r, j) for every
 * logical block j < nblk(r): the per-(request, block) items every later call walks,
 * so one launch per layer covers the whole batch (Tutti 阅读笔记, 伪代码 1
 * retrieve_layer and the note after it: the CPU launches the I/O kernel once per
 * layer, O(L) not O(L x blocks)).  Validates each request (counts >= 0, required
 * pointers non-null, 16-byte alignment), every pool block id (in [0, N)), every
 * full-block id of a hit block (in [0, hit_src_blocks)) and, if check_injective,
 * that no pool block id repeats.
 * The plan also describes each request's strided row sources (hit rows, miss rows)
 * by tensor maps, built on the device from templates that the host encodes with the
 * driver's cuTensorMapEncodeTiled (looked up through the runtime on the first plan
 * call; host work only, nothing allocated), when their strides lay the rows out
 * without overlap (each stride at least the extent below it) and some dimension spans
 * at least 1 MiB; the copy
 * calls then read a segment of rows of one source (a whole segment, or the rows a
 * block has left after its whole segments) with one tiled bulk-tensor load instead
 * of one bulk load per row.  The maps span exactly the rows a request
 * declares: T_hit rows of a full block without a table, all B token rows of each
 * of the hit_src_blocks blocks with a table (so with a table every one of those
 * blocks must be whole), and T_miss rows of the miss KV, each over all L layers.
 * Sources without maps (or a driver without the encoder) are read one bulk load per
 * row: the results are the same bytes either way.
 *   geom            host pointer
 *   d_reqs          device array of n_req requests (caller-owned, read only; may be
 *                   NULL when n_req == 0)
 *   d_block_tables  device int32 tables, packed in request order (read only; may be
 *                   NULL when n_req == 0)
 *   d_plan          device buffer of plan_bytes >= kvl_plan_bytes(geom, n_req) bytes,
 *                   16-byte aligned, caller-owned; overwritten.  The plan resolves
 *                   every item's addresses and block ids when it is built: later
 *                   edits to the requests or tables take effect only through a new
 *                   plan.  The copy calls update the plan's claim counters, so two
 *                   calls on one plan for the same layer and op must not overlap on
 *                   the GPU (calls for different layers or ops may).
 * Device-side status: EINVAL (detail = first bad request), EALIGN (detail = first bad
 * request), ERANGE (detail = smallest bad work item, or the item count when it
 * exceeds N), EDUP (detail = smallest repeated block id).  The largest code wins. */
kvl_status kvl_batch_plan(const kvl_geom *geom, int32_t n_req, const kvl_request *d_reqs,
                          const int32_t *d_block_tables, int32_t check_injective,
                          void *d_plan, size_t plan_bytes, void *stream);

/* kvl_batch_plan_static_scratch -- kvl_batch_plan for callers that cannot allocate
 * device memory.  The pages have no counterpart to this call.
 * Some callers cannot call cudaMalloc: for instance an inference engine whose own
 * allocator owns all of the HBM (its KV pool took it up front), where an extra
 * scratch allocation would fail or break the engine's accounting.  This call needs
 * no scratch from the caller: the injectivity bitmap lives in a fixed device array
 * inside libkvl.so (KVL_STATIC_SCRATCH_POOL_BLOCKS / 8 bytes = 512 KiB, held by
 * every GPU that loads the library until the process exits).  The caller still
 * passes the requests, the block tables and the plan, and the plan needs only
 * kvl_plan_layout(...)[8] bytes (everything before the bitmap section); the plan it
 * writes is the same as kvl_batch_plan's and the copy calls accept it.
 * It allocates nothing: no cudaMalloc, no cudaFree, no allocating library routine.
 * The array's device address belongs to the CUDA context the library's module was
 * loaded into.  Every call that is not being captured into a graph looks it up again
 * (cudaGetSymbolAddress, with the device current) and remembers it with the current
 * context's id; a call made while `stream` is capturing uses that remembered address
 * only if the current context is the one it was taken in, and otherwise returns
 * KVL_ECUDA with nothing launched.  So make one call on the device, outside capture,
 * before capturing one, and again after a cudaDeviceReset or a context switch.
 * Limits and sharing: pool_blocks above KVL_STATIC_SCRATCH_POOL_BLOCKS returns
 * KVL_EINVAL and launches nothing.  Every call on a device shares the one array,
 * which keeps the last call's contents; each call clears the bits it uses before
 * using them.  Calls that overlap on the GPU (other streams, other host threads)
 * race on the array in both directions: one call's bits can make another report a
 * duplicate that is not there, and one call's clearing can erase another's bits, so
 * a real duplicate can pass with KVL_OK and the copy calls would then give one pool
 * block two writers.  Serialise such calls.  Other arguments, checks and status
 * codes are those of kvl_batch_plan. */
#define KVL_STATIC_SCRATCH_POOL_BLOCKS (1 << 22)
kvl_status kvl_batch_plan_static_scratch(const kvl_geom *geom, int32_t n_req,
                                         const kvl_request *d_reqs, const int32_t *d_block_tables,
                                         int32_t check_injective, void *d_plan, size_t plan_bytes,
                                         void *stream);

/* The copy calls below work on the layers [layer, layer + layer_count) in one launch:
 * layer_count = 1 is the layer-wise pipeline of the pages (one launch per layer, as
 * soon as that layer's data exists); a larger count serves callers that have several
 * layers ready, e.g. restoring a whole prefix (Tutti 阅读笔记, 伪代码 1 and its note:
 * the I/O kernel is loaded once per layer, O(L) launches, not O(L x blocks)).
 * layer >= 0, layer_count >= 1, layer + layer_count <= L, pool_blocks * layer_count
 * < 2^31; otherwise KVL_EINVAL.  `launch` may be NULL (the whole GPU, no flags); a
 * negative max_ctas, an unknown flag or both host flags together is KVL_EINVAL.
 * d_plan is a plan built for this geom, and plan_bytes the size of the buffer at d_plan
 * (the plan_bytes the plan was built with, or the bytes a static-scratch plan needs).
 * plan_bytes below kvl_plan_layout(geom, 0)[8], the smallest plan of this geometry,
 * returns KVL_EINVAL and launches nothing, so no kernel reads past a buffer the host
 * knows to be too small.  The kernels read nothing of the plan beyond plan_bytes: a
 * plan whose recorded request count needs more than plan_bytes (a buffer sized for
 * fewer requests than the plan in it holds), or that was built for other arrays or
 * another geometry (L, P, B, Rp or N), is refused on the device (KVL_EINVAL in its
 * status) before any of its n_req-sized sections is read.
 * d_reqs and d_block_tables are the arrays the plan was built from; NULL only if it was
 * built from NULL (a batch of no requests); other NULLs are refused on the device. */

/* kvl_slice_layer -- hit_layer[l] = hit_full_block[:, l] for every request
 * (DualPath KV Loading, "Dual-Path Loading": objects table and the slice_layer step
 * of pe_read_path / de_read_path).  Writes, for each layer of the launch, sum(T_hit)
 * rows of R bytes to d_hit_out (device, caller-owned): launch layer i (= l - layer) at
 * row i*sum(T_hit) + hit_off[r] + t. */
kvl_status kvl_slice_layer(const kvl_geom *geom, const void *d_plan, size_t plan_bytes,
                           const kvl_request *d_reqs, int32_t layer, int32_t layer_count,
                           void *d_hit_out, const kvl_launch *launch, void *stream);

/* kvl_merge_scatter_paged -- slice, concatenate and scatter in one pass:
 * complete_layer[l] = hit_layer[l] rows then miss_layer[l] rows (DualPath KV Loading,
 * pe_read_path concatenate_tokens; de_read_path merge_layer), and token t of plane p
 * goes to pool block table[t / B], slot t % B (Tutti 阅读笔记, 前置知识 3, eq. (2)).
 *   d_pool          device pool [L][P][N][B][Rp], caller-owned; the slots of the
 *                   launch's layers named by the tables are written
 *   d_complete_out  NULL, or device memory that also receives complete_layer[l]:
 *                   launch layer i at row i*sum(T_all) + tok_off[r] + t, R bytes each */
kvl_status kvl_merge_scatter_paged(const kvl_geom *geom, const void *d_plan, size_t plan_bytes,
                                   const kvl_request *d_reqs, const int32_t *d_block_tables,
                                   int32_t layer, int32_t layer_count, void *d_pool,
                                   void *d_complete_out, const kvl_launch *launch, void *stream);

/* kvl_gather_layer_objects -- per-layer K/V objects <-> paged blocks.
 * direction KVL_GATHER: object (l, p, j) = pool block table[j] of plane p, layer l,
 * for every request: the 2*nblk objects of a layer ready for transfer (Tutti
 * 阅读笔记, 前置知识 5 eq. (4); the worked trace's 8,000 per-layer entries for 4,000
 * blocks).  direction KVL_SCATTER_BACK: the inverse, restoring objects into their
 * paged blocks (伪代码 1 retrieve_layer).  Each request's `objects` must be non-NULL. */
kvl_status kvl_gather_layer_objects(const kvl_geom *geom, const void *d_plan, size_t plan_bytes,
                                    const kvl_request *d_reqs, const int32_t *d_block_tables,
                                    int32_t layer, int32_t layer_count, void *d_pool,
                                    int32_t direction, const kvl_launch *launch, void *stream);

/* kvl_read_status -- copy the plan's status word and its detail to the host.
 * Synchronises `stream` first, so it reports every call enqueued before it.
 * code/detail may be NULL.  Returns KVL_ECUDA if the copy fails, else KVL_OK. */
kvl_status kvl_read_status(const void *d_plan, int32_t *code, int64_t *detail, void *stream);

/* kvl_diag_wait_timeout -- exercise the copy kernels' bounded wait.  Launches one
 * warp that waits, with the same bounded mbarrier wait the copy kernels use, for 16
 * bytes that nothing delivers; after limit_us microseconds (1 .. 10^7) it gives up and
 * writes KVL_ETIMEOUT to *d_status (device int32), then releases the barrier itself.
 * It copies nothing.  Used to check that a wait that runs out returns an error the
 * host can read and leaves the context usable. */
kvl_status kvl_diag_wait_timeout(int32_t limit_us, int32_t *d_status, void *stream);

/* ---------------------------------------------------------------------------
 * The 8-bit paged cache: pages of codes of one byte with a float32 scale for each
 * (page, head), who writes them (kvl_cache_append), who reads them (kvl_attend), the
 * rotary positions of their keys (kvl_rotary) and who owns them (kvl_pages_*).
 *
 * Codes are laid out as a pool of the copy calls above with P = 2 and Rp = H*d bytes,
 * scales as one with B = 1 and Rp = 4*H, both indexed by the same page ids, so slices,
 * merge-scatters, gathers and scatter-backs persist and restore both parts of a page:
 *   code of (layer l, plane p, page b, slot s, head h, element e):
 *       codes  + ((((l*2 + p)*N + b)*B + s)*H + h)*d + e       (p: 0 = K, 1 = V)
 *   scale of (l, p, b, h):  scales[((l*2 + p)*N + b)*H + h]
 *   value = code * scale.
 *
 * Device-side problems are recorded in a report (KVL_REPORT_BYTES of device memory,
 * 16-byte aligned, prepared by kvl_report_reset and read by kvl_read_status): the
 * offending sequence (page, pair) is left out, everything else is done, nothing traps.
 * Unlike a plan's status a report does not hold later calls back.  A NULL report
 * records nothing.  detail = the batch entry (or pair) with the smallest number.
 * ------------------------------------------------------------------------- */
#define KVL_REPORT_BYTES 256
#define KVL_CODE_FLOAT 0 /* 8-bit float: 4 exponent bits, 3 mantissa bits, +-448, NaN, no infinity */
#define KVL_CODE_INT 1   /* signed 8-bit integer, -127 .. 127 */
#define KVL_TYPE_BFLOAT 0
#define KVL_TYPE_HALF 1
#define KVL_TYPE_FLOAT 2

typedef struct kvl_cache {
    int32_t n_layers;     /* L */
    int32_t n_kv_heads;   /* H */
    int32_t head_dim;     /* d: a multiple of 16, at most 256 */
    int32_t block_tokens; /* B: tokens per page, any */
    int64_t pool_blocks;  /* N: pages */
    int32_t code_type;    /* KVL_CODE_FLOAT or KVL_CODE_INT */
    int32_t reserved;     /* 0 */
    void *codes;          /* [L][2][N][B][H][d], 16-byte aligned */
    float *scales;        /* [L][2][N][H] */
} kvl_cache;

/* A batch of sequences (host struct, device arrays).  Entry i of the batch is the
 * sequence of slot slots[i] (or slot i): its pages are table entries
 * tables[slot*table_stride ...] (or, with table_offsets, tables[table_offsets[slot]] up
 * to table_offsets[slot + 1], e.g. a plan's blk_off and its packed tables), it holds
 * lens[slot] tokens and its fresh tokens, the last of those it holds, are the rows
 * starts[i] .. starts[i + 1] of the call's row arrays. */
typedef struct kvl_sequences {
    int32_t n_seq;   /* batch entries */
    int32_t n_slots; /* rows of lens (and of tables) */
    int64_t n_rows;  /* rows of the row arrays: starts[n_seq] is at most this */
    int64_t table_stride;
    const int32_t *tables;
    const int64_t *table_offsets; /* NULL, or n_slots + 1 */
    const int32_t *lens;          /* n_slots */
    const int32_t *slots;         /* NULL, or n_seq */
    const int32_t *starts;        /* n_seq + 1 */
} kvl_sequences;

/* Rows of heads: element e of head h of row t is at data + t*row_stride + h*head_stride
 * + e*(element size); strides in bytes, everything a multiple of 16 bytes.  So q, k and v
 * may be parts of one fused projection's rows. */
typedef struct kvl_rows {
    void *data;
    int64_t row_stride;
    int64_t head_stride;
} kvl_rows;

/* Prepare a report: no problem recorded. */
kvl_status kvl_report_reset(void *d_report, void *stream);

/* Rotary positions.  The first 2*n_freq elements of a head are n_freq pairs: (i, i + n_freq),
 * or (2i, 2i + 1) when interleaved; pair i of a row at position p turns by the angle
 * p * inv_freq[i]: a' = gain*(a cos - b sin), b' = gain*(b cos + a sin).  The elements
 * after the pairs are copied.  Scaling for long contexts is in inv_freq and gain
 * (kvl_rotary_frequencies).  The angle is reduced exactly, however long the context. */
typedef struct kvl_rope {
    const float *inv_freq; /* device, n_freq */
    int32_t n_freq;        /* 2*n_freq <= head_dim */
    int32_t interleaved;   /* 0 or 1 */
    float gain;            /* 1, or the attention gain of a scaled context */
    int32_t reserved;      /* 0 */
} kvl_rope;

/* kvl_rotary -- turn n_sets tensors (at most 4, e.g. q and k; src[i] -> dst[i], which may
 * be the same memory with the same strides and must not otherwise overlap) of n_rows rows
 * by their positions, in one launch.  inverse != 0 applies the transposed map: the
 * gradient of the inputs from that of the outputs.  src, dst and n_heads are host arrays
 * of n_sets; positions is a device array of n_rows int32.  head_dim: a multiple of 8
 * (of 4 for KVL_TYPE_FLOAT) up to 512; n_freq a multiple of 4. */
kvl_status kvl_rotary(const kvl_rope *rope, int64_t n_rows, int32_t head_dim, int32_t type,
                      const int32_t *positions, int32_t n_sets, const kvl_rows *src,
                      const kvl_rows *dst, const int32_t *n_heads, int32_t inverse, void *stream);

/* Frequencies of n_freq pairs (host arrays, host work): inv_freq[i] = base^(-i/n_freq), then
 *   KVL_ROPE_PLAIN       nothing more
 *   KVL_ROPE_LINEAR      divided by factor (positions interpolated)
 *   KVL_ROPE_BASE        base *= factor^(n_freq/(n_freq - 1)): the slowest pair slows by factor
 *   KVL_ROPE_WAVELENGTH  pairs that turn fewer than `low` times over trained_context tokens
 *                        slow by factor, those that turn more than `high` times stay, a
 *                        linear join in the number of turns between them
 * *gain receives 1, or with scale_gain != 0 the logarithmic gain 0.1*ln(factor) + 1. */
#define KVL_ROPE_PLAIN 0
#define KVL_ROPE_LINEAR 1
#define KVL_ROPE_BASE 2
#define KVL_ROPE_WAVELENGTH 3
kvl_status kvl_rotary_frequencies(int32_t kind, double base, int32_t n_freq, double factor,
                                  double low, double high, double trained_context,
                                  int32_t scale_gain, float *inv_freq, float *gain);

/* kvl_cache_append -- quantise the batch's fresh K and V rows into their pages of one layer.
 * Fresh token t of entry i (row starts[i] + t) takes cache position lens - (fresh tokens) + t.
 * For each page and head that receives rows x, with qmax 448 (float) or 127 (int):
 *   scale' = max(scale, max|x| * (1/qmax), 1e-30) in 32 bits, where the old scale counts only if the page's
 *            first fresh slot is not slot 0 (the page held tokens before);
 *   codes of the slots before the fresh ones become round(code * (scale / scale'));
 *   a fresh element's code is round(clamp(x * (1/scale'))), to nearest, ties to even.
 * max|x| is over finite elements; an infinity takes the largest code of its sign, a NaN
 * the NaN code (float) or 0 (int).  With a rope (NULL: none) K is turned by its cache
 * position first, in 32 bits; its n_freq is a multiple of 8 (kvl_rotary, which takes multiples
 * of 4, can turn other keys beforehand).  Pages of different entries that receive rows must differ
 * (kvl_pages_extend sees to it).  type: of the rows, KVL_TYPE_*. */
kvl_status kvl_cache_append(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs,
                            int32_t type, const kvl_rows *k, const kvl_rows *v,
                            const kvl_rope *rope, void *d_report, void *stream);

/* kvl_attend -- attention of the batch's fresh rows over their sequences' cached tokens (the
 * fresh ones among them).  Fresh row t of an entry stands at position p = lens - (fresh rows)
 * + t; query head h reads KV head h / (n_heads / H).  With s_j = sm_scale * (q . K_j):
 *   visible: 0 <= j < lens, j <= p if causal, j > p - window if window > 0;
 *   out = sum_j softmax(s)_j V_j,  lse = log(sum_j exp(s_j)) (natural, optional).
 * A row that sees nothing, or only scores of -infinity, gets out = 0 and lse = -infinity.  Cached
 * bytes that no row sees (slots past lens, pages past the sequence's end) are never part of a
 * result, whatever they hold.
 * Statistics and sums are held in 32 bits.  A token's probability times its V scale enters the
 * product as a half: right to 2^-11 of itself, or to 2^-29 of the largest such product of the row.
 * Scales are taken to be finite and at least 0 (one that is NaN, where a row sees it, makes the
 * row's out and lse NaN).  A V scale of at most 1e-30, that of a page of zeros, counts as 2^-80.  A
 * token's part is lost where its probability times its V scale is below 2^-126 of the largest such
 * product of the row (so none above 2^-30 of the largest probability while V scales are at most 2^16).
 * n_rows * (n_heads / H) is below 2^31 - 256.  A call with more work than 2^31 groups of 16 tokens
 * (about 10^10 tokens, counted for each KV head and row tile) does nothing and the report says
 * KVL_ERANGE.
 *   max_new   0, or a bound on the fresh rows of any entry that the caller knows; it chooses
 *             kernels, so results depend on it in their rounding only */
typedef struct kvl_attention {
    kvl_rows q;       /* n_rows rows of n_heads heads */
    kvl_rows out;     /* likewise; must not overlap q */
    float *lse;       /* NULL, or [n_rows][n_heads] */
    int32_t n_heads;  /* a multiple of n_kv_heads */
    int32_t type;     /* KVL_TYPE_BFLOAT or KVL_TYPE_HALF, of q and out */
    float sm_scale;
    int32_t causal;   /* 0 or 1 */
    int32_t window;   /* 0: none; > 0 needs causal */
    int32_t max_new;
} kvl_attention;

/* Device memory kvl_attend needs for one call (0 for a bad cache); it holds partial results
 * of a row split over several CTAs.  The first KVL_ATTEND_ZERO_BYTES have to be zero before
 * the first call and are zero again after every call; calls that may run at the same time
 * need a workspace each. */
#define KVL_ATTEND_ZERO_BYTES 16384
size_t kvl_attend_workspace_bytes(const kvl_cache *cache);
/* The number of the stream capture that `stream` is in, unique in the process; 0: none.  Zeroing a
 * workspace inside a capture happens when the graph runs and not before: such a workspace belongs to
 * that graph alone. */
uint64_t kvl_capture_id(void *stream);
kvl_status kvl_attend(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs,
                      const kvl_attention *attn, void *d_workspace, size_t workspace_bytes,
                      void *d_report, void *stream);

/* kvl_attend_shared -- attention of a batch whose sequences share prefixes, as forks do: the same results as
 * kvl_attend, but the tokens that a group of entries shares are read once for the rows of all of them.
 *   groups   entries groups[g] .. groups[g + 1] of the batch are group g (ascending; entries outside all groups
 *            share nothing, a group may be empty)
 *   tokens   the first tokens[g] tokens of every sequence of group g are in the same pages: those of the group's
 *            first sequence are read.  (After kvl_pages_fork and _extend that holds of a parent's whole
 *            pages; a partly filled last one is replaced by copies.)
 * Every row sees all shared tokens: tokens[g] is at most lens - (fresh rows) of each entry with rows.  An entry for
 * which it is more is left out, its rows not written, and reported (KVL_ERANGE with its number); so are the
 * entries of a group that is bad: reported with the group's number, KVL_EINVAL for its range, KVL_ERANGE for
 * more shared tokens than its first sequence holds.  Where groups or starts descend (reported, KVL_EINVAL), or the
 * kernel of the shared tokens gives up (KVL_ETIMEOUT), no entry that shares tokens is written; where starts
 * descend, others may be left out too.  A group whose first sequence is bad, or whose first or last start is out of
 * range, is left out with it.
 * A call with a window, without groups, or whose entries may have more than KVL_SHARED_ROWS rows (max_new, without
 * one n_rows, times n_heads / H), reads every entry's own table, as kvl_attend does.
 * d_workspace is kvl_attend's; d_parts (16-byte aligned; not looked at by such a call) needs no preparation and
 * holds nothing between calls.  A call's launches pass data through it, so calls that may run at the same time, or are
 * made by host threads at the same time on one stream, need one each. */
#define KVL_SHARED_ROWS 40
typedef struct kvl_shared {
    int32_t n_groups; /* at most 1048576 */
    int32_t reserved; /* 0 */
    const int32_t *groups; /* device, n_groups + 1 */
    const int32_t *tokens; /* device, n_groups */
} kvl_shared;

size_t kvl_attend_shared_parts_bytes(const kvl_cache *cache, int32_t n_seq, int32_t n_groups, int64_t n_rows,
                                     int32_t n_heads);
kvl_status kvl_attend_shared(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs,
                             const kvl_shared *shared, const kvl_attention *attn, void *d_workspace,
                             size_t workspace_bytes, void *d_parts, size_t parts_bytes, void *d_report,
                             void *stream);

/* kvl_weigh -- how much attention each cached token received: for every token j that an entry's sequence holds,
 *   mass_out[slot][j] = mass_in[slot][j] + sum over fresh rows t and query heads h that see j of
 *                       exp(sm_scale * (q_th . K_j) - lse_th)
 * with rows, visibility and sm_scale as kvl_attend's and lse as it returned them, so each term is the probability
 * that row t's head h gave token j.  q enters the products as halves under a power of two, one for each row or, where
 * entries have more than 16 rows, one for 128 rows beside each other, of whose largest finite element what is below 2^-39
 * is lost.  With begin != 0 the fresh tokens' mass_in counts as 0 (a step's first call;
 * the layers after it add).  A row whose lse is infinite gives nothing.  mass_out may be mass_in; entries without
 * fresh rows, and what lies past a sequence's tokens, are not written.  Slots of a call must differ.  Sums are in
 * 32 bits and come out the same every time.  A sequence longer than a row of masses is left out (KVL_ERANGE).
 * Where starts descend (reported, KVL_EINVAL), entries beside the bad one may be left out too.
 * Scales are taken to be finite.  d_workspace (16-byte aligned) needs no preparation and holds nothing between
 * calls; calls need one each as with d_parts above.  kvl_weigh_workspace_bytes is 0 for bad arguments. */
typedef struct kvl_weighing {
    kvl_rows q;             /* n_rows rows of n_heads heads */
    const float *lse;       /* [n_rows][n_heads] */
    const float *mass_in;   /* [n_slots][in_stride] */
    float *mass_out;        /* [n_slots][out_stride] */
    int64_t in_stride, out_stride;
    int64_t tokens;         /* that a row of masses has room for (at most the strides, but for one slot) */
    int32_t n_heads;        /* a multiple of n_kv_heads */
    int32_t type;           /* KVL_TYPE_BFLOAT or KVL_TYPE_HALF, of q */
    float sm_scale;
    int32_t causal;         /* 0 or 1 */
    int32_t window;         /* 0: none; > 0 needs causal */
    int32_t max_new;        /* 0, or a bound on the fresh rows of any entry; chooses kernels */
    int32_t begin;          /* 0 or 1 */
    int32_t reserved;       /* 0 */
} kvl_weighing;

size_t kvl_weigh_workspace_bytes(const kvl_cache *cache, int32_t n_seq, int64_t n_rows, int32_t n_heads,
                                 int32_t max_new);
kvl_status kvl_weigh(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs,
                     const kvl_weighing *weighing, void *d_workspace, size_t workspace_bytes, void *d_report,
                     void *stream);

/* Page bookkeeping, all of it in device memory, without a host in the loop.
 * refs[b] counts the table entries of live sequences that name page b (0: free); slot s
 * holds lens[s] tokens in the pages tables[s*table_stride ...], ceil(lens[s] / B) of them;
 * entries past those mean nothing.  Which page is taken is a function of the state alone:
 * always the free pages with the lowest numbers. */
typedef struct kvl_pages {
    int64_t pool_blocks;  /* N */
    int32_t block_tokens; /* B */
    int32_t n_slots;      /* at most 1048576 */
    int64_t table_stride; /* entries per slot: a sequence holds at most this many pages */
    int32_t *tables;
    int32_t *lens;
    int32_t *refs;        /* N */
    int32_t *pairs;       /* [N][2] page copies to make: (from, to), 8-byte aligned */
    int32_t *n_pairs;     /* their number */
} kvl_pages;

/* kvl_pages_extend -- slots[i] (n of them, distinct) will hold counts[i] more tokens.  Entry by
 * entry, in order: if the sequence's last page is partly filled and was shared when the call
 * began, it is replaced by a free page (pairs receives (old, new), to be copied by
 * kvl_pages_copy before the tokens are appended); then the further pages it needs follow.
 * Pages are handed out lowest number first; lens, tables and refs follow.  If the free pages
 * (pages freed by this call do not count) or a table row's entries are not enough for the
 * whole batch, nothing is changed, n_pairs is 0 and the report says KVL_ERANGE.  One call gives
 * one sequence at most 1048576 pages. */
kvl_status kvl_pages_extend(const kvl_pages *pages, int32_t n, const int32_t *slots,
                            const int32_t *counts, void *d_report, void *stream);

/* kvl_pages_fork -- children[i] becomes a copy of parents[i]: same length, same pages, each
 * with one more reference.  A child must be empty (length 0), named once, and no parent. */
kvl_status kvl_pages_fork(const kvl_pages *pages, int32_t n, const int32_t *parents,
                          const int32_t *children, void *d_report, void *stream);

/* kvl_pages_free -- the sequences of slots[0 .. n) end: length 0, one reference less on each of
 * their pages.  An empty slot stays as it is. */
kvl_status kvl_pages_free(const kvl_pages *pages, int32_t n, const int32_t *slots,
                          void *d_report, void *stream);

/* kvl_pages_compact -- move the live pages to the numbers below their count n_live: the k-th
 * live page numbered n_live or more (in order) goes to the k-th free number below n_live.
 * tables (of every slot) and refs are rewritten, pairs receives the copies to make. */
kvl_status kvl_pages_compact(const kvl_pages *pages, void *d_report, void *stream);

/* kvl_pages_copy -- copy the pages of pairs[0 .. *d_n_pairs) (device; at most max_pairs of
 * them), codes and scales of every layer, from pair[0] to pair[1].  Sources and destinations
 * must be disjoint and destinations distinct, as extend and compact leave them. */
kvl_status kvl_pages_copy(const kvl_cache *cache, const int32_t *pairs, const int32_t *d_n_pairs,
                          int64_t max_pairs, void *d_report, void *stream);

/* kvl_pages_evict -- shorten slots[i] (n of them, distinct) to keep[i] tokens.  A sequence that holds no more stays
 * as it is.  Else it keeps its first f = min(first, keep) tokens, its last r = min(recent, keep - f) and, of
 * those between, the keep - f - r of the largest mass; of equal masses the first ones, a NaN counting as less
 * than any number, and all as equal where mass is NULL.  The kept tokens stay in order: the k-th becomes token
 * k.  Its masses move along, and the rest of its row of masses becomes 0.  Pages before f / B stay; the tokens from there on go
 * to fresh pages (the lowest free numbers, in batch order), whose codes kvl_tokens_move brings before anything
 * else is done to the pages, and the pages they were in lose a reference.
 * If a slot is bad (KVL_EINVAL), named twice (KVL_EDUP) or too long for its table or masses, or there are too few
 * free pages (pages freed by this call do not count; KVL_ERANGE with detail n), nothing is changed.
 * Its launches pass data through `moves` to each other and to kvl_tokens_move: no other eviction into the same
 * `moves` comes between, from another host thread or stream.
 * A key keeps the rotary position it was turned by, while attention counts positions from the
 * sequence's shortened start: later keys are turned by their own positions before they are appended. */
typedef struct kvl_eviction {
    const int32_t *keep;  /* device, n */
    float *mass;          /* NULL, or [n_slots][mass_stride] */
    int64_t mass_stride;
    int64_t tokens;       /* that a row of masses has room for (at most the stride, but for one slot) */
    int32_t first;
    int32_t recent;
} kvl_eviction;

/* What an eviction asks to be moved (device arrays, written by kvl_pages_evict). */
typedef struct kvl_moves {
    int32_t *from; /* [N][B][2]: (page, slot) of each token of a fresh page; a page of -1: none; 8-byte aligned */
    int32_t *to;   /* [N]: the fresh pages */
    int32_t *at;   /* [n_slots + 1]: where each entry's begin in `to` */
    int32_t *n;    /* their number */
} kvl_moves;

kvl_status kvl_pages_evict(const kvl_pages *pages, int32_t n, const int32_t *slots, const kvl_eviction *eviction,
                           const kvl_moves *moves, void *d_report, void *stream);

/* kvl_tokens_move -- bring the codes of an eviction's tokens, all layers, K and V: for each fresh page and head
 *   scale' = the largest scale of the pages that its tokens come from,
 *   code'  = round(code * (scale / scale')) in 32 bits, to nearest, ties to even; tokens whose scale is scale'
 *            keep their codes.
 * Slots of a page that receive no token are not written.  max_pages: pages that `to` has room for. */
kvl_status kvl_tokens_move(const kvl_cache *cache, const kvl_moves *moves, int64_t max_pages, void *d_report,
                           void *stream);

/* Human-readable name of a status code (static string). */
const char *kvl_status_string(kvl_status s);

/* Kernel launches one call of each entry point makes (for launch accounting):
 * which = 0 plan, 1 slice, 2 merge-scatter, 3 gather / scatter-back, 4 rotary, 5 append,
 * 6 attend (at most), 7 pages extend, 8 fork, 9 free, 10 compact, 11 copy, 12 attend_shared (at
 * most), 13 weigh (at most), 14 evict, 15 tokens move. */
int32_t kvl_launches_per_call(int32_t which);

#ifdef __cplusplus
}
#endif

#endif /* KVL_H */
