/*
 * ula.h -- C ABI of the PB-LRU KV residency engine for MI355X (gfx950).
 *
 * The engine implements, for one GPU in data-parallel form, the residency
 * layer described in "UlaCache: Unified Logical Addressing for Sparse LLM
 * Serving" (paper-daily.com summary):
 *
 *  - Section 2: the serving engine allocates and selects KV entries by fixed
 *    logical address only; the library decides whether the GPU pool or the
 *    host pool holds each entry, moves it, and keeps a logical->physical
 *    mapping table. In DP mode an entry lives in exactly one of the two
 *    pools. Layers that share one sparse selection look up and de-duplicate
 *    it once per layer group.
 *  - Section 3: the GPU pool is managed by PB-LRU: slots are labelled with the
 *    scheduling round that last touched them (per layer group, a ring of round
 *    buckets and one cold bucket, each a bitmap with summaries); victims come
 *    from free slots, then cold, then older ring buckets, never the running
 *    round's bucket. Rows move before the mapping changes, the completion
 *    signal comes last, and readers wait for it.
 *
 * Conventions
 *  - Every layer group g in [0, num_groups) has its own GPU pool of
 *    gpu_slots slots, host pool of host_slots slots, mapping table over
 *    logical addresses [0, logical_capacity), and replacement state.
 *  - A slot holds the rows of all layers_per_group layers of one logical
 *    entry; a row is row_bytes opaque bytes (FP8 latent, rope and scales in
 *    the pages' model; never interpreted here).
 *  - Mapping table encoding (uint32): s < 2^31 = GPU slot s; 0x80000000|h =
 *    host slot h; 0xFFFFFFFF = never appended.
 *  - Bucket bitsets: words of 32 bits, slot s is bit (s & 31) of word
 *    (s >> 5); order free, cold, ring[0] .. ring[B-1].
 *  - All calls that take a stream enqueue work on that HIP stream
 *    (hipStream_t passed as uint64_t; 0 = null stream) and return without
 *    waiting, unless stated otherwise. Device-side errors of an enqueued call
 *    are reported by the next ula_sync.
 *
 * Ownership
 *  - The caller allocates and owns the device workspace (ula_device_bytes
 *    bytes, 256-byte aligned, device memory) and the pinned host pool
 *    (ula_host_bytes bytes, page-locked and device-mapped, e.g. from
 *    ula_host_alloc), the selection and output buffers and the streams. They
 *    must outlive all work enqueued on them. The library owns only the
 *    opaque context and the layout inside the two buffers.
 *
 * Errors
 *  - Every call returns ULA_OK (0) or a negative code. Errors detected on the
 *    host are returned at once and change nothing. Errors detected on the
 *    device during an enqueued step are latched per group and the remaining
 *    kernels of that step exit before changing any state; errors a gather
 *    detects are latched per group in a separate word that steps do not read,
 *    so a gather never stops a step part-way. The next ula_sync returns the
 *    first latched code and the context becomes unusable (ULA_ESTATE) for every
 *    call but ula_export_state, ula_read_rows, ula_sync and ula_destroy.
 *  - ULA_ECAPACITY is detected before any state changes, so an exported state
 *    after it is the state before the failed step.
 *
 * Threading: a context belongs to one host thread. Groups are independent and
 * may be driven on different streams; calls on one group must be ordered. The
 * groups share one host link, so once steps arrive on more than one stream the
 * library orders each step's host-link launch after the previous step's (of any
 * group) with an event; the rest of one group's step (lookup, swap, gathers)
 * still runs beside another group's host-link launch. A gather issued on a
 * stream other than its step's must be ordered after the step (an event, or a
 * stream wait on ula_flag_address). The library orders what comes after it:
 * the group's next launch that moves rows out of GPU slots (the next step's
 * swap, an append under ULA_PLACE_RING, a release) waits, by events, for the
 * group's gathers enqueued since its last such launch, on any stream; the next
 * step's lookup, marking and host-link transfers do not wait and may run beside
 * those gathers (each step resolves its selection into one of two buffers, by
 * step parity, and a gather reads its step's). HIP places a process's streams
 * on a few hardware queues, each running its launches in order: with more step
 * streams than queues, one group's lookup can wait behind another group's
 * gathers, so many groups run best on two step streams (groups alternating)
 * with the gathers on a third.
 */
#ifndef ULA_H
#define ULA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  ULA_OK = 0,
  ULA_EINVAL = -1,       /* bad argument or configuration */
  ULA_ERANGE = -2,       /* logical address outside [0, N) or never appended */
  ULA_EDUP = -3,         /* append of an address already appended, or twice in one call */
  ULA_EHOSTFULL = -4,    /* no free GPU or host slot left for an append */
  ULA_ECAPACITY = -5,    /* a step selects more distinct entries than the GPU pool holds */
  ULA_ENOTRESIDENT = -6, /* gather before its step completed, or of an entry not on the GPU */
  ULA_ESTATE = -7,       /* the context was poisoned by an earlier device error */
  ULA_EHIP = -8,         /* a HIP runtime call failed; ula_strerror gives its text */
  ULA_EBUSY = -9,        /* ula_init_static: this device's static workspace is held by a live context */
  ULA_ETOOBIG = -10      /* ula_init_static: the configuration needs more than the static workspace */
};

typedef struct ula_ctx ula_ctx;

typedef struct {
  int32_t num_groups;        /* layer groups, each with its own pools and state, >= 1 */
  int32_t layers_per_group;  /* layers sharing one selection, >= 1 */
  int32_t row_bytes;         /* bytes per row, multiple of 16, <= 4096 */
  int32_t ring_buckets;      /* B >= 1 ring buckets (plus one cold and one free bucket) */
  int32_t logical_capacity;  /* N: logical addresses [0, N), 1 <= N < 2^31 */
  int32_t gpu_slots;         /* P >= 1 GPU slots per group */
  int32_t host_slots;        /* H >= 0 host slots per group, P + H < 2^31 */
  int32_t max_sets;          /* most selection sets per step */
  int32_t max_k;             /* most entries per selection set; max_sets * max_k < 2^31 */
  int32_t max_append;        /* most addresses staged per append chunk, >= 1 */
  int32_t policy;            /* ULA_POLICY_PBLRU (0, default) or ULA_POLICY_LRU (1) */
  int32_t placement;         /* where ula_append puts new entries: ULA_PLACE_LOWEST (0, default)
                                or ULA_PLACE_RING (1, PB-LRU only) */
} ula_config;

/* Placement of appended entries (section 2: the library decides which pool holds
 * new KV; the pages do not say how).
 *  - ULA_PLACE_LOWEST: in list order each entry takes the lowest free GPU slot,
 *    joining the cold bucket, else the lowest free host slot; appends never
 *    evict (with a full GPU pool, new entries start in the host pool and come
 *    in through a step's miss path when selected).
 *  - ULA_PLACE_RING: new entries count as used in the current round (section 3:
 *    recent entries stay on the GPU): in list order each entry takes the next
 *    slot of the step's victim order (free ascending, then cold, then ring
 *    buckets oldest to newest, never the current bucket) and joins the current
 *    bucket; an entry displaced from that slot moves, rows and all, to the
 *    lowest free host slot; when no such slot is left, entries take the lowest
 *    free host slots. The current bucket is that of the group's last step. */
enum { ULA_PLACE_LOWEST = 0, ULA_PLACE_RING = 1 };

/* Replacement policies. PB-LRU is the pages' policy (UlaCache summary, section 3).
 * Exact LRU is the standard policy the pages compare it against (sections 3 and 4):
 * one timestamp per GPU slot (a hit or a load at step t sets it to t; an
 * appended slot s counts as s - P, so older than any step and ordered by slot)
 * and a scan of the whole pool each step; victims are the free slots in
 * ascending order, then the occupied slots by (timestamp, slot), never a slot
 * stamped with the current step. Everything else (lookup, pairing, data moves,
 * commit, signal, appends) is shared. */
enum { ULA_POLICY_PBLRU = 0, ULA_POLICY_LRU = 1 };

typedef struct {
  int64_t unique;     /* distinct valid addresses selected by the step */
  int64_t hits;       /* of those, already on the GPU */
  int64_t misses;     /* of those, brought in from the host pool */
  int64_t evictions;  /* misses whose victim slot held an entry (sent to the host) */
  int64_t from_free;  /* misses that took a free GPU slot */
  int64_t invalid;    /* -1 padding entries in the selection */
} ula_step_stats;

typedef struct {             /* caller-allocated host buffers filled by ula_export_state */
  uint32_t* map;             /* [N] mapping table */
  int32_t* gown;             /* [P] owner logical address of each GPU slot, -1 = empty */
  int32_t* hown;             /* [H] owner logical address of each host slot, -1 = empty */
  uint32_t* bitsets;         /* [(B + 2)][ceil(P / 32)]: free, cold, ring[0..B-1]; under exact
                                LRU only the free set is kept (the others read as empty) */
  int32_t cur;               /* current ring bucket */
  int64_t flag;              /* last completed step (completion counter) */
  ula_step_stats last;       /* statistics of that step */
  int32_t* stamps;           /* nullable, [P]: exact LRU timestamps (appended slot s: s - P,
                                free slot: 0); under PB-LRU left untouched */
} ula_state_host;

/* Bytes of device workspace / pinned host pool a configuration needs; 0 for an
 * invalid configuration (section 2: in DP mode each GPU has one GPU pool and one
 * host pool; here every layer group has its own of each, plus its mapping table
 * and replacement state in the workspace). Pure host functions (no device is
 * touched). */
size_t ula_device_bytes(const ula_config* cfg);
size_t ula_host_bytes(const ula_config* cfg);

/* Lay out the workspace, initialise every group (nothing appended, all GPU slots
 * free, all host slots free, cur = 0, flag = 0) on `stream`, and return a context
 * (section 2: the pools and the mapping table; section 3: one ring plus a cold
 * bucket per layer group).
 * dev_ws: device memory of ula_device_bytes(cfg) bytes, 256-byte aligned.
 * host_pinned: pinned, device-mapped host memory of ula_host_bytes(cfg) bytes
 * (may be NULL when host_slots == 0). Errors: ULA_EINVAL, ULA_EHIP. */
int ula_init(const ula_config* cfg, void* dev_ws, void* host_pinned, uint64_t stream,
             ula_ctx** out);

/* ula_init for callers that cannot allocate device memory (code that must not
 * call hipMalloc or a caching allocator: tight serving loops, harnesses that
 * forbid allocation). Exactly ula_init, with the device workspace taken from a
 * static array the library holds on every device it runs on (32 MiB per device,
 * kept until the process ends) instead of a dev_ws argument: the current
 * device's array, resolved once per device. Only a configuration with
 * ula_device_bytes(cfg) <= 32 MiB fits (ULA_ETOOBIG otherwise, nothing
 * touched). One live context per device may hold the array: another call on the
 * same device before that context's ula_destroy returns ULA_EBUSY (two contexts
 * on one array would overwrite each other's state). Every call starts from a
 * fully initialised workspace whatever an earlier context left in it.
 * The call allocates no device memory and no pinned host memory (the context
 * itself is ordinary host memory; host_pinned is still the caller's pool). Such
 * a context has no pinned staging buffers: ula_append of more than 128 entries
 * (256 under ULA_POLICY_LRU) runs in chunks whose addresses travel by value in
 * the launches, host-resident rows are copied in and waited for chunk by chunk,
 * and ula_release copies its addresses from the caller's memory and waits for
 * that copy before it returns; the events
 * of step timing and of the ordering of host-link launches across streams are
 * created by the call that first needs them. Everything else behaves as for a
 * context from ula_init.
 * Errors: ULA_EINVAL, ULA_ETOOBIG, ULA_EBUSY, ULA_EHIP. */
int ula_init_static(const ula_config* cfg, void* host_pinned, uint64_t stream, ula_ctx** out);

/* Append n new logical entries to group g (section 2: the library decides the
 * pool), placed as the configuration's placement says: by default, in list
 * order each entry takes the lowest free GPU slot (joining the cold bucket) or,
 * when none is free, the lowest free host slot, and appends never evict; under
 * ULA_PLACE_RING each entry joins the current bucket, displacing entries to the
 * host pool (see above). la_host: n addresses in host memory. rows: n x layers_per_group x
 * row_bytes bytes, packed, in device memory (rows_on_device = 1) or host memory
 * (rows_on_device = 0); rows must stay valid until the stream reaches the call.
 * An append of more than 128 entries (256 under ULA_POLICY_LRU), or of
 * host-resident rows, copies its
 * addresses through one of four pinned staging buffers of the group: with all
 * four still in use by enqueued appends, the call first waits for the oldest to
 * be consumed (the host runs at most four such appends ahead of the device).
 * Validated on the host first: ULA_EINVAL (bad g or n < 0), ULA_ERANGE (address
 * outside [0, N)), ULA_EDUP (already appended or repeated), ULA_EHOSTFULL (not
 * enough free slots in total); nothing changes on error. */
int ula_append(ula_ctx* ctx, int32_t group, int32_t n, const int32_t* la_host,
               const void* rows, int32_t rows_on_device, uint64_t stream);

/* Release n finished entries of group g (a request has ended; section 1: in a
 * shared pool the space one request frees serves the others). Each address must
 * be appended and listed once; it becomes absent and may be appended again. Its
 * GPU slot leaves whatever bucket holds it and joins the free slots, which later
 * steps take first for their misses and appends take before host slots; or its
 * host slot joins the free host slots. The ring, the current bucket, the
 * completion counter and the statistics do not change. Staged evicted rows of
 * the last step are written to the host pool first (a released host slot may be
 * waiting for one). Gathers of the last step's selection after a release resolve
 * through the mapping table (a released entry is then ULA_ERANGE). la_host: n
 * addresses in host memory. Enqueued on `stream`, ordered after the group's
 * earlier calls like ula_append.
 * Validated on the host first: ULA_EINVAL (bad g or n < 0), ULA_ERANGE (address
 * outside [0, N) or not appended), ULA_EDUP (repeated), ULA_ESTATE; nothing
 * changes on error. */
int ula_release(ula_ctx* ctx, int32_t group, int32_t n, const int32_t* la_host, uint64_t stream);

/* Copy the n entries at addresses src .. src + n - 1 of group g to the new
 * addresses dst .. dst + n - 1 (a request that forks, in a beam or for several
 * samples: sections 1 and 2, one shared pool, placement is the library's):
 * exactly ula_append of the destination addresses, in ascending order, with the
 * sources' rows, whichever pool holds them; the rows never pass through the host
 * program. Sources stay as they are (under ULA_PLACE_RING an append may move one
 * to the host pool, as any entry). The new entries belong to no step yet: select
 * them in the next one, or gather them before it through the mapping table
 * (ULA_ENOTRESIDENT if they were placed in the host pool). Enqueued on `stream`,
 * ordered after the group's earlier calls like ula_append; not in a graph
 * capture (ULA_EINVAL).
 * Validated on the host first: ULA_EINVAL (bad g or n < 0), ULA_ERANGE (an address
 * outside [0, N), or a source not appended), ULA_EDUP (a destination already
 * appended, so also ranges that overlap), ULA_EHOSTFULL (not enough free slots in
 * total), ULA_ESTATE; nothing changes on error. */
int ula_fork(ula_ctx* ctx, int32_t group, int32_t src, int32_t dst, int32_t n, uint64_t stream);

/* Give the n entries at addresses src .. src + n - 1 of group g the addresses dst
 * .. dst + n - 1 (section 2: the table maps addresses to places; here only the
 * table and the owner words change, no row moves): compaction of the address
 * space after releases. The ranges may overlap, as in memmove; a destination
 * must be absent or one of the sources. Slots, buckets, timestamps, the
 * completion counter and the statistics do not change. Gathers of the last step's
 * selection afterwards resolve through the mapping table (an old address is then
 * ULA_ERANGE or another entry). Enqueued and ordered like ula_fork.
 * Validated on the host first: ULA_EINVAL, ULA_ERANGE (an address outside [0, N),
 * or a source not appended), ULA_EDUP (a destination taken by another entry),
 * ULA_ESTATE; nothing changes on error. */
int ula_rename(ula_ctx* ctx, int32_t group, int32_t src, int32_t dst, int32_t n, uint64_t stream);

/* One decode step (one scheduling round) of group g over n_sets x k selected
 * addresses (device memory, row-major, -1 = padding), section 3: de-duplicate
 * (first occurrence in row-major order) and look up once for the group; advance
 * the ring and fold the reused bucket into cold; move hits into the current
 * bucket; pick one victim per miss (free, cold, ring oldest -> newest, ascending
 * slot inside a bucket, never the current bucket); bring the missed rows in from
 * the host pool; then update the mapping table and owners and raise the
 * completion counter to the step number. Data path: the missed rows are read
 * into device memory in the same launch that marks the hits and plans the
 * victims; the victims' rows are staged in device memory as the missed rows
 * replace them; the staged rows reach the host slots their misses vacated
 * during the group's next step, beside that step's reads from the host (a miss
 * of a row evicted by the previous step reads its staged copy), or when
 * ula_read_rows or ula_release needs the host pool current. So the mapping
 * table can name a host slot for an evicted entry one step before its rows
 * land there; every GPU reader is unaffected (a row in the host pool is read
 * only by a later step of the group, which writes the staged rows first or
 * reads the staged copy). Enqueued on
 * `stream` with no host synchronisation.
 * Host errors: ULA_EINVAL (bad g, n_sets > max_sets, k > max_k, negative sizes),
 * ULA_ESTATE. Device errors (reported by ula_sync): ULA_ERANGE, ULA_ECAPACITY. */
int ula_step(ula_ctx* ctx, int32_t group, int32_t n_sets, int32_t k, const int32_t* sel_dev,
             uint64_t stream);

/* One decode step of group g with its appends (section 2: the new positions a
 * step produces are appended, then the step selects among all entries):
 * exactly ula_append(ctx, group, n_app, la_host, rows, rows_on_device, stream)
 * followed by ula_step(ctx, group, n_sets, k, sel_dev, stream), with the same
 * arguments, placement and results, in fewer launches: an append of at most 128
 * entries (256 under ULA_POLICY_LRU; and at most max_append) with rows in device
 * memory runs in the
 * step's first launch, beside the de-duplication, which does not read the
 * mapping table; other appends run as ula_append does, before the step.
 * n_app = 0 is a plain step. Both parts are validated on the host before
 * anything is enqueued: any host error of ula_append or ula_step is returned
 * with nothing changed. Device errors of the step are reported by ula_sync as
 * for ula_step; the appended entries stay appended. */
int ula_append_step(ula_ctx* ctx, int32_t group, int32_t n_app, const int32_t* la_host,
                    const void* rows, int32_t rows_on_device, int32_t n_sets, int32_t k,
                    const int32_t* sel_dev, uint64_t stream);

/* Gather layer `layer` of every selected entry of group g into out_dev
 * (device memory, n_sets x k x row_bytes bytes, packed; a -1 entry gives a zero
 * row). Reads the GPU pool through the mapping table after checking that the
 * group's completion counter equals the group's last step (section 3: readers
 * wait for the signal); call it once per layer of the group, or gather several
 * layers in one launch with ula_gather_layers. On a stream other
 * than the step's, order it after the step first (event, or a stream wait on
 * ula_flag_address reaching the step number): the counter check inside the
 * gather is a relaxed read that only catches a gather that runs before the
 * counter is raised (ULA_ENOTRESIDENT); the rows of an unordered gather that
 * finds the counter raised are undefined, since nothing orders its reads after
 * the step's writes on another cache. The group's later calls need no
 * ordering after the gather: the library makes the next launch that moves rows
 * out of GPU slots wait for it (see Threading). A gather that runs while the
 * group's next step fails on the device may find that step's error and write
 * nothing (ula_sync reports the error); an address appended, forked or renamed
 * only after the step resolves through the mapping table (an error if the entry is
 * not on the GPU), and is undefined if that call runs beside the gather.
 * Host errors: ULA_EINVAL, ULA_ESTATE, ULA_ENOTRESIDENT (no step yet).
 * Device errors (reported by ula_sync): ULA_ENOTRESIDENT (counter not reached,
 * or an entry not on the GPU), ULA_ERANGE. */
int ula_gather(ula_ctx* ctx, int32_t group, int32_t layer, int32_t n_sets, int32_t k,
               const int32_t* sel_dev, void* out_dev, uint64_t stream);

/* Gather layers layer0 .. layer0 + n_layers - 1 of every selected entry of
 * group g in one launch (section 2: the layers of a group share one selection,
 * and the later layers are fetched while an earlier one is in use). out_dev
 * (device memory) holds n_layers per-layer buffers one after the other, each
 * n_sets x k x row_bytes bytes laid out as ula_gather writes it: the result is
 * exactly that of ula_gather(layer0 + i, out_dev + i * n_sets * k * row_bytes)
 * for each i. Since a slot keeps its layers side by side, each entry's layers
 * are read as one contiguous run. Same checks and errors as ula_gather, plus
 * ULA_EINVAL unless 0 <= layer0, 1 <= n_layers and layer0 + n_layers <=
 * layers_per_group. */
int ula_gather_layers(ula_ctx* ctx, int32_t group, int32_t layer0, int32_t n_layers, int32_t n_sets,
                      int32_t k, const int32_t* sel_dev, void* out_dev, uint64_t stream);

/* ---- Operators on the rows' contents ------------------------------------
 * The calls above move rows as opaque bytes. The ones below read or write what
 * is in them, in one of two formats with values in e4m3 (OCP 8-bit floating
 * point, 4 exponent and 3 fraction bits, no infinities) and fp32 scales
 * (section 4: the KV cache is held in FP8). Integers and floats are stored
 * little-endian, in this order and without gaps:
 *
 *  ULA_ROWS_LATENT, 656 bytes: 512 latent channels e4m3 | 64 rotary channels
 *    bf16 | 4 scales fp32, one per 128 latent channels. One token per entry; one
 *    representation serves every query head (section 1).
 *      key   = [latent channel x its scale (512), rotary channels (64)]
 *      value = [latent channel x its scale (512)]
 *  ULA_ROWS_HEADS: keys e4m3 [kv_heads][block_tokens][head_dim] | values e4m3,
 *    the same shape | key scales fp32 [kv_heads] | value scales fp32 [kv_heads]
 *    | int32 tokens of the block in use, 0..block_tokens (outside that range it
 *    counts as the nearest end) | zeros up to a multiple of 16 bytes. An entry
 *    is a block of block_tokens tokens with one scale per head for its keys and
 *    one for its values; tokens behind the count are never used. Query heads
 *    are shared evenly: head h reads KV head h / (heads / kv_heads). */
enum { ULA_BF16 = 0, ULA_FP16 = 1, ULA_FP32 = 2 };
enum { ULA_ROWS_LATENT = 0, ULA_ROWS_HEADS = 1 };

typedef struct {
  int32_t kind;              /* ULA_ROWS_LATENT or ULA_ROWS_HEADS */
  int32_t kv_heads;          /* heads rows: >= 1 (latent rows: this and the next two are not read) */
  int32_t head_dim;          /* heads rows: 64 or 128 */
  int32_t block_tokens;      /* heads rows: 1, 2, 4, 8 or 16 */
} ula_row_format;

/* Bytes of one row (one layer of one entry) of a format, a multiple of 16; 0 for
 * an invalid one or one that is longer than 4096 bytes, the most a row can be. */
size_t ula_row_format_bytes(const ula_row_format* rows);

/* Rotary positions. Of R rotated channels, pair i (0 <= i < R / 2) turns by the
 * angle pos[axis(i)] * theta^(-2i / R): (x0, x1) becomes (x0 cos - x1 sin,
 * x0 sin + x1 cos). Pair i is channels (i, i + R / 2), or (2i, 2i + 1) if
 * interleaved. The first sections[0] pairs go by the first axis, the next
 * sections[1] by the second, the rest by the third (for text one axis; for images
 * and video two or three, such as time, height, width). Positions are int32,
 * negative ones too; angles are computed in 64 bits. */
typedef struct {
  int32_t axes;              /* 1, 2 or 3 */
  int32_t sections[3];       /* pairs of each axis, >= 0; those of the axes in use sum to R / 2 */
  int32_t interleaved;       /* 0 or 1 */
  double theta;              /* base, finite and > 0 */
} ula_rotary;

typedef struct {
  ula_row_format rows;
  int32_t type;              /* of the inputs: ULA_BF16, ULA_FP16 or ULA_FP32 */
  int32_t n;                 /* entries */
  int32_t layers;            /* rows per entry */
  const void* a;             /* latent rows: latent channels [n][layers][512]
                                heads rows: keys [n][layers][block_tokens][kv_heads][head_dim] */
  const void* b;             /* latent rows: rotary channels [n][layers][64]
                                heads rows: values, shaped as the keys */
  int64_t a_stride[4];       /* strides in elements: entry, layer, then (heads rows) token, head; */
  int64_t b_stride[4];       /*   the last dimension is contiguous */
  const int32_t* positions;  /* nullable (nothing turns): [n][axes], heads rows [n][block_tokens][axes], packed */
  const int32_t* count;      /* heads rows, nullable (all in use): tokens in use of each entry, [n] */
  ula_rotary rotary;         /* read if positions is given; turns the rotary channels, or whole keys */
} ula_pack_args;

/* Write n x layers rows in the given format to rows_dev (device memory, packed,
 * 16-byte aligned: what ula_append takes as device rows). scale = max(amax / 448,
 * 2^-126) over each scale's values (heads rows: over the tokens in use; the
 * others' codes are 0), code = value / scale rounded to nearest even. An infinity
 * takes the largest code and a NaN the NaN code; neither enters amax. Rotary
 * channels are turned in 32 bits and rounded to bf16 once. A pure function of its
 * device inputs: nothing of an engine is involved, and it may be captured into a
 * graph. Errors: ULA_EINVAL (null pointer, n or layers < 0, unknown type, invalid
 * format or rotary, misaligned pointers, 2^26 rows or more, or heads rows of 2^34
 * keys' elements or more), ULA_EHIP. */
int ula_pack_rows(const ula_pack_args* args, void* rows_dev, uint64_t stream);

typedef struct {
  int32_t type;              /* of x and out: ULA_BF16, ULA_FP16 or ULA_FP32 */
  int32_t n, heads, dim;     /* tokens, heads, channels of a head: even, 2..256, all turned */
  int32_t inverse;           /* 1: turn back, which is also the gradient of the turn */
  const void* x;             /* [n][heads][dim], last dimension contiguous */
  void* out;                 /* the same shape; x itself with the same strides, or no overlap;
                                its own rows share no elements (ULA_EINVAL if a stride says so) */
  int64_t x_stride[2];       /* strides in elements: token, head */
  int64_t out_stride[2];
  const int32_t* positions;  /* [n][axes] packed */
  ula_rotary rotary;
} ula_rotate_args;

/* Turn the heads of n tokens (the rotary part of queries, or its way back) by
 * their positions; each result is rounded to its type once. A pure function of
 * its device inputs; it may be captured into a graph. Errors: ULA_EINVAL (also
 * more rows than a launch takes: n * heads < 2^25 always fits), ULA_EHIP. */
int ula_rotate(const ula_rotate_args* args, uint64_t stream);

typedef struct {
  int32_t type;              /* of q, k and the results: ULA_BF16, ULA_FP16 or ULA_FP32 */
  int32_t n, dim;            /* tokens; channels of a head: even, 2..256 */
  int32_t q_heads, k_heads;  /* either may be 0 */
  int32_t rotary_dim;        /* R: the first channels, which turn: even, 0..dim (0: norms alone) */
  int32_t weight_type;       /* of the weights: type or ULA_FP32 */
  float eps;                 /* 2^-126 .. 2^96 */
  const void* q;             /* [n][q_heads][dim], last dimension contiguous */
  const void* k;             /* [n][k_heads][dim] */
  void* q_out;               /* the same shapes; q and k themselves with the same strides, or no overlap with */
  void* k_out;               /*   anything else; rows share no elements (ULA_EINVAL if a stride says so) */
  int64_t q_stride[2];       /* strides in elements: token, head */
  int64_t k_stride[2];
  int64_t q_out_stride[2];
  int64_t k_out_stride[2];
  const void* q_weight;      /* [dim], nullable (all 1) */
  const void* k_weight;
  const int32_t* positions;  /* [n][axes] packed, read if rotary_dim > 0 */
  ula_rotary rotary;         /* of R channels, read if rotary_dim > 0 */
} ula_norm_args;

/* Norms of the queries and keys of n tokens, each head by itself, and their turn in
 * the same pass: y_i = w_i x_i / sqrt(mean of x^2 + eps) over the head's channels,
 * then the first R channels turned as by ula_rotate. In 32 bits, rounded to the type
 * once; rows of large values do not overflow; a row with an infinity gives 0 and NaN in its
 * place, one with a NaN gives NaN. A pure function of its device inputs; it may be
 * captured into a graph. Errors: ULA_EINVAL (also more rows than a launch takes:
 * n * (q_heads + k_heads) < 2^25 always fits), ULA_EHIP. */
int ula_norm_rotate(const ula_norm_args* args, uint64_t stream);

typedef struct {
  ula_row_format rows;       /* the group's rows; its bytes must equal the configuration's row_bytes */
  int32_t type;              /* of q and out: ULA_BF16 or ULA_FP16 */
  int32_t heads;             /* query heads, >= 1; heads rows: a multiple of kv_heads */
  float scale;               /* factor of the logits, finite (times log2(e) too) */
  const void* q;             /* [n_sets][heads][576 (latent) or head_dim], last dimension contiguous */
  int64_t q_set_stride;      /* strides in elements */
  int64_t q_head_stride;
  void* out;                 /* [n_sets][heads][512 (latent) or head_dim], last dimension contiguous */
  int64_t out_set_stride;
  int64_t out_head_stride;
  float* lse;                /* nullable, [n_sets][heads] packed: ln of the sum of exp(logits) */
  void* workspace;           /* device memory of ula_attend_bytes bytes, 16-byte aligned; may be NULL for 0 */
  size_t workspace_bytes;
} ula_attend_args;

/* Bytes of workspace that ula_attend needs for these sizes (0: none, or an
 * invalid argument, which ula_attend reports). A pure host function. */
size_t ula_attend_bytes(const ula_row_format* rows, int32_t n_sets, int32_t k, int32_t heads);

/* Attention of every selection set's queries over its selected entries of layer
 * `layer` of group g, read from the GPU pool where they lie (introduction:
 * attention reads only the selected KV rows; section 3: after the completion
 * signal):
 *   logit_j = scale * q . key_j,  out = sum_j softmax(logit)_j value_j
 * over the entries j of the set (every token in use of each entry for heads
 * rows). -1 entries contribute nothing; a set with nothing else gives out = 0
 * and lse = -inf. An address listed more than once counts as often. Sums, the
 * softmax and the products' accumulators are in 32 bits; keys enter exactly,
 * softmax weights times value scales are rounded to fp16 before the second
 * product (2^-11 of each, or 2^-32 of the set's largest; for fp16 results what that
 * leaves goes through another: 2^-22 of each; value scales are meant to lie between
 * 2^-60 and 2^80: smaller ones count as 2^-60 in that largest, and with larger ones
 * small weights are lost), results once to the type of out. A logit
 * that is NaN or +infinity makes that head's outputs and log-sum NaN; an entry of
 * logit -infinity has no weight, and a set with no other gives 0 and -inf. No
 * unselected row is ever read. The order of the sums depends on the sizes alone, so
 * the same call gives the same bits.
 * Results split over several workgroups are joined through the workspace, which
 * belongs to the call until the stream has run it: calls that may run at the
 * same time need workspaces of their own. q, out, lse and the workspace must not
 * overlap, nor rows of out (ULA_EINVAL if one of its strides says so). q and out
 * rows whose pointer and strides keep them 16-byte aligned are read and written in
 * vectors, others element by element.
 * Which entries, streams and errors: as for ula_gather (the selection is looked
 * up through the group's last step where it is that step's, else through the
 * mapping table; on another stream the call must be ordered after the step; the
 * library orders the group's later row moves after it). It may not be captured
 * into a graph, since the step it belongs to is fixed at the call: ULA_EINVAL.
 * Host errors: ULA_EINVAL (also n_sets * heads >= 2^24, heads > 2^16, latent rows
 * with k > 2^21, heads rows with k * block_tokens >= 2^30, or a launch of 2^23
 * workgroups, which n_sets * heads * (1 + k / 2048) < 2^22 never makes), ULA_ESTATE,
 * ULA_ENOTRESIDENT (no step yet), ULA_EHIP. Device errors (reported by ula_sync):
 * ULA_ENOTRESIDENT, ULA_ERANGE; an entry with such an error counts as padding. */
int ula_attend(ula_ctx* ctx, int32_t group, int32_t layer, int32_t n_sets, int32_t k,
               const int32_t* sel_dev, const ula_attend_args* args, uint64_t stream);

typedef struct {
  ula_attend_args attend;    /* of one node: strides of sets and heads; lse is [n_sets][nodes][heads] packed,
                                q, out, the workspace and the rest as for ula_attend */
  int32_t nodes;             /* drafted tokens of each set, 1..64 */
  int64_t q_node_stride;     /* strides in elements: q and out are [n_sets][nodes][heads][...] */
  int64_t out_node_stride;
  const void* drafts;        /* the drafted tokens' rows, packed as ula_pack_rows writes them, 16-byte aligned:
                                [n_sets][ceil(nodes / block_tokens)][layers_per_group] rows (latent rows: a
                                token a block) */
  const uint64_t* visible;   /* [n_sets][nodes]: bit j says that the node sees drafted token j */
} ula_tree_args;

/* Bytes of workspace that ula_attend_tree needs (0: none, or an invalid argument,
 * which ula_attend_tree reports). A pure host function. */
size_t ula_attend_tree_bytes(const ula_row_format* rows, int32_t n_sets, int32_t k, int32_t nodes, int32_t heads);

/* Attention of a tree of drafted tokens over the cache (section 4: a step verifies
 * tokens that a draft model proposed): every node of a set attends to the set's
 * selected entries, as in ula_attend, and to those drafted tokens whose bit its mask
 * has (its ancestors and itself, as a rule). The drafted tokens' rows come from the
 * caller: nothing is appended before they are accepted. Selected rows are read once
 * for all nodes of a set. Drafted token j of a set is token j % block_tokens of its
 * block j / block_tokens; tokens behind a block's count, and bits from `nodes` on, are
 * never used. A node that sees nothing, in a set with nothing selected, gives 0 and
 * -inf. A drafted token's row reaches only the nodes that see it, whatever it holds: one
 * with a NaN code among its latent channels or its values, or a value scale (latent
 * rows: a scale) that is not finite, makes the heads that see it NaN, log-sums too (heads
 * rows: so does a value scale of a selected entry). Heads rows' value scales below 2^-80
 * count as 0, and the largest product of weight and scale is that of the scales as they
 * are. Softmax weights times value scales go through in two fp16 parts for bf16 results
 * too (2^-22 of each, or 2^-32 of the set's largest). The rest (formula, other roundings,
 * order of the sums, which entries, streams, errors) is as for ula_attend; drafts and visible may be read until the stream has run the call.
 * Host errors: also ULA_EINVAL
 * for nodes outside 1..64, null or misaligned drafts (16 bytes) or visible (8 bytes), rows
 * of out that share elements (each stride is looked at), n_sets * nodes * heads >= 2^24
 * or nodes * heads > 2^16. */
int ula_attend_tree(ula_ctx* ctx, int32_t group, int32_t layer, int32_t n_sets, int32_t k, const int32_t* sel_dev,
                    const ula_tree_args* args, uint64_t stream);

typedef struct {
  ula_row_format rows;       /* the group's rows; its bytes must equal the configuration's row_bytes */
  int32_t type;              /* of q: ULA_BF16 or ULA_FP16 */
  int32_t nodes, heads;      /* query rows of a set: nodes (1 without a tree, at most 64) x heads */
  float scale;               /* factor of the logits, as in the attention */
  const void* q;             /* [n_sets][nodes][heads][576 (latent) or head_dim], last dimension contiguous */
  int64_t q_set_stride;      /* strides in elements */
  int64_t q_node_stride;     /* not read for one node */
  int64_t q_head_stride;
  const float* lse;          /* [n_sets][nodes][heads] packed, from the attention */
  float* shares;             /* nullable, [n_sets][k] packed */
  int64_t* scores;           /* nullable, [logical_capacity]; one of the two is required */
} ula_weigh_args;

/* The softmax weight that each selected entry got in an attention with these queries
 * and log-sums, summed over the set's query rows:
 *   share_j = sum_r exp(scale * q_r . key_j - lse_r)
 * (heads rows: over an entry's tokens in use and over every head with its KV head), written to
 * shares and added to the score of the entry's address (eviction by accumulated
 * attention weight: see ula_lightest). Scores are whole numbers in units of 2^-32, so an address that
 * is listed more than once gets the same score whatever the order of the adds. -1
 * entries have share 0 and add nothing. What the score was is not looked at: one that ula_lightest has
 * set to -1, weighed again before its address is released (by another layer), is there again for
 * the next choice. So all layers are weighed before a choice that marks, or its addresses' scores set to
 * -1 once more after the last of them. A row whose lse is not finite counts for
 * nothing (it attended to nothing; a rejected node is left out that way). With log-sums
 * that cover more than these entries (a tree's drafted tokens) shares are of the whole.
 * A share that is NaN adds nothing to the score, one above 2^22 adds that; a score holds
 * 2^31 of weight, so a program that runs on for so long halves its scores before. Products, logits and
 * sums are in 32 bits, summed in an order that depends on the sizes alone. Nothing but keys
 * is read of the rows. q, lse, shares and scores must not overlap. Calls that add to the same scores at the
 * same time are fine. Which entries, streams and errors: as for ula_attend. Host errors: also
 * ULA_EINVAL for nodes outside 1..64, nodes * heads > 2^16, n_sets * nodes * heads >= 2^24, and heads rows
 * with n_sets * k * block_tokens >= 2^30. */
int ula_weigh(ula_ctx* ctx, int32_t group, int32_t layer, int32_t n_sets, int32_t k, const int32_t* sel_dev,
              const ula_weigh_args* args, uint64_t stream);

typedef struct {
  int64_t* scores;           /* device memory, [capacity], 8-byte aligned; read, and written if mark */
  int32_t capacity;          /* scores there are */
  int32_t ranges;            /* ranges of addresses */
  const int32_t* first;      /* host memory, [ranges] each: addresses first .. last - 1, */
  const int32_t* last;
  const int32_t* count;      /*   and how many entries each gives up, 0..most */
  int32_t most;              /* columns of out */
  int32_t mark;              /* 1: the scores of the entries chosen become -1 */
  int32_t* out;              /* device memory, [ranges][most] */
  void* workspace;           /* device memory of ula_lightest_bytes bytes, 32-byte aligned; may be NULL for 0 */
  size_t workspace_bytes;
} ula_lightest_args;

/* Bytes of workspace that ula_lightest needs for these ranges (0: none, or invalid
 * arguments, which ula_lightest reports). A pure host function. */
size_t ula_lightest_bytes(const ula_lightest_args* args);

/* Of each range of addresses the `count` entries of least score (eviction by
 * accumulated attention weight; a request's first tokens and its recent ones stay out
 * of its range), ties by lowest address, in ascending order of address: what
 * ula_release takes, once copied to the host. Entries of negative score are not there:
 * absent addresses, which the caller, or mark, set to -1 (ula_weigh adds to those as to any). Where a range has fewer, and from
 * `count` on, out is -1. Ranges may be empty, and may overlap unless mark is set.
 * Nothing of an engine is involved; calls that may run at the same time need workspaces of
 * their own. It may be captured into a graph (the ranges are those of the call; the
 * host arrays are read before it returns).
 * Errors: ULA_EINVAL (null or misaligned pointers, negative sizes, first > last, a count outside
 * 0..most, ranges * most >= 2^31, overlapping ranges with mark, a missing or small
 * workspace), ULA_ERANGE (an address outside [0, capacity)), ULA_EHIP. */
int ula_lightest(const ula_lightest_args* args, uint64_t stream);

/* Wait for `stream`, then report the first latched device error of any group
 * (poisoning the context) or ULA_OK (section 3: a host waiter for the steps'
 * completion). per_group_out (nullable, num_groups entries) receives each
 * group's last step statistics (section 4: the GPU hit rate is hits over
 * distinct selected entries). Errors: ULA_EINVAL, ULA_EHIP, or the latched code. */
int ula_sync(ula_ctx* ctx, uint64_t stream, ula_step_stats* per_group_out);

/* Copy group g's canonical state (mapping table, owners, bucket bitsets, the
 * current bucket, the completion counter and the last step's statistics) into
 * caller host buffers, after synchronising the device. Staged evicted rows stay
 * staged: none of these fields depends on the host pool's bytes. Works on a
 * poisoned context. cur is derived from the counter (the ring advances once
 * per step, section 3), not read from the device. Errors: ULA_EINVAL (null
 * context or buffers, bad group), ULA_EHIP. */
int ula_export_state(ula_ctx* ctx, int32_t group, ula_state_host* out);

/* Read back the stored rows (all layers, layers_per_group x row_bytes bytes
 * each) of n appended entries of group g into host memory, from whichever pool
 * holds them (for checks of stored data; no passage of the pages behind it) (writes any staged evicted rows to the host pool and synchronises
 * the device first). ULA_ERANGE if an address was never
 * appended. */
int ula_read_rows(ula_ctx* ctx, int32_t group, int32_t n, const int32_t* la_host,
                  void* out_host);

/* Device address of group g's completion counter (int64, equals the last
 * completed step), for hipStreamWaitValue64 on another stream (section 3:
 * readers wait for the completion signal). A step that fails on the device
 * leaves the last completed step in the counter and sets bit 62, so a stream
 * waiting for the counter to be greater than or equal to that step's number is
 * released rather than left waiting; a gather it then issues is refused, and
 * ula_sync reports the failure. ula_export_state reports the counter without
 * that bit. */
int ula_flag_address(ula_ctx* ctx, int32_t group, void** dev_ptr);

/* Timing, off by default; ula_set_timing takes an OR of these flags (ULA_EINVAL
 * for unknown bits).
 *  - ULA_TIMING_STEP: events between the phases of every step. ula_read_timing
 *    gives, for the last step of group g, in milliseconds: [0] lookup +
 *    de-duplication, [1] hit marking + fold + victim selection, with the missed
 *    rows read in and the previous step's evicted rows written out over the
 *    host link in the same launch, [2] rows into the victim slots + commit +
 *    signal. It synchronises on the step's last event.
 *  - ULA_TIMING_GATHER: every gather launch records events in its own dispatch,
 *    so their interval is the kernel's execution alone (no launch overhead).
 *    ula_read_gather_timing synchronises on them and returns the summed kernel
 *    time and the number of launches since the last read (then resets both).
 *  - ULA_TIMING_LINK: the same for every step's host-link launch (the launch
 *    that reads the missed rows in and writes the previous step's evicted rows
 *    out while it marks hits and selects victims; under exact LRU, the first
 *    select pass, which carries that work); read by ula_read_link_timing.
 * Errors: ULA_EINVAL (unknown flag, null pointer, step timing never switched
 * on), ULA_EHIP. */
enum { ULA_TIMING_STEP = 1, ULA_TIMING_GATHER = 2, ULA_TIMING_LINK = 4 };
int ula_set_timing(ula_ctx* ctx, int32_t flags);
int ula_read_timing(ula_ctx* ctx, int32_t group, float* ms_out3);
int ula_read_gather_timing(ula_ctx* ctx, double* kernel_ms, int64_t* launches);
int ula_read_link_timing(ula_ctx* ctx, double* kernel_ms, int64_t* launches);

/* Release the context (not the caller's buffers). Waits for no stream.
 * Resource management only; no passage of the pages behind it. */
int ula_destroy(ula_ctx* ctx);

/* Text of an error code (also the last HIP error text for ULA_EHIP). Plumbing;
 * no passage of the pages behind it. */
const char* ula_strerror(int code);

/* Pinned, device-mapped host memory for the host pool (hipHostMalloc);
 * NULL on failure. ula_host_free returns ULA_OK or ULA_EHIP. Plumbing (section
 * 2's host pool lives in it). */
void* ula_host_alloc(size_t bytes);
int ula_host_free(void* p);

#ifdef __cplusplus
}
#endif

#endif /* ULA_H */
