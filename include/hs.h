/*
 * hs.h -- C ABI of a GB300-native (sm_103a) HiSparse swap-in resolution library.
 *
 * HiSparse (paper abstract, "HiSparse: Turbocharging Sparse Attention with
 * Hierarchical Memory") keeps each request's full KV history in host memory and
 * bounds its decode footprint with a small, fixed-size GPU cache; a fused CUDA kernel
 * resolves each layer's top-k selections -- hit detection, LRU replacement and
 * host-to-device fetches -- inside the decode CUDA graph. The blog commentary
 * (sections two and three) adds that the same step updates the page table and that a
 * hit is used in place while a miss is swapped in over an LRU-chosen victim.
 *
 * One hs_ctx is one layer's cache for num_requests requests. It owns:
 *   host KV store   pinned + mapped host memory, [R][C] rows of hs_host_stride() bytes
 *                   (the first entry_bytes of each row are the entry);
 *   device buffer   HBM, [R][S] rows of entry_bytes bytes;
 *   page table      int32 [R][C] in HBM: position -> slot, -1 when not resident;
 *   slot tokens     int32 [R][S]: slot -> position, -1 when empty;
 *   last use        int32 [R][S]: per-slot recency stamp, -1 when never used;
 *   step            int32 [R]: calls made so far per request (the stamp of the next call);
 *   a miss area (miss lists and the flags that let the two kernels of a call
 *   overlap) and a device status word (internal).
 * R = num_requests, C = context_len, S = slots. Everything starts empty: page
 * table, slot tokens and last use at -1, step 0, device buffer zero.
 *
 * Replacement rule (the pages leave the order open; this is the deterministic
 * reading implemented, HS_POLICY_LRU, the default; hs_set_policy selects the FIFO and
 * random comparison policies): in a call with stamp t, slots hit by the selection are
 * stamped t and are not evictable; the distinct missed positions, in ascending
 * order, take in order the non-hit slots with the smallest (last_use, slot index);
 * the position a victim held is unmapped, the new one mapped and stamped t, and its
 * host row copied into the slot. A negative selection is padding (slot -1, neither
 * hit nor miss); a selection >= C (in a pooled context, >= the request's extent
 * length) yields slot -1 and sets HS_STATUS_RANGE; a position
 * repeated within one row resolves to the same slot each time, counts once, and sets
 * HS_STATUS_DUP.
 *
 * Error convention: functions returning int return HS_OK (0) or a negative HS_ERR_*;
 * hs_last_error() then describes the failure (per calling thread). Device-side input
 * problems never trap: they set bits of the status word (hs_get_status).
 * Threading: calls on one hs_ctx must not overlap on the GPU (state is per context);
 * different contexts are independent.
 */
#ifndef HS_H_
#define HS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct hs_ctx hs_ctx;
/* A CUDA stream (cudaStream_t); NULL is the legacy default stream. */
typedef struct CUstream_st* hs_stream_t;
/* A CUDA event (cudaEvent_t). */
typedef struct CUevent_st* hs_event_t;

#define HS_OK 0
#define HS_ERR_INVALID (-1) /* bad argument; nothing was enqueued */
#define HS_ERR_CUDA (-2)    /* a CUDA runtime call failed */
#define HS_ERR_NOMEM (-3)   /* host or device allocation failed */
#define HS_ERR_LIMIT (-4)   /* sizes beyond what this build supports */

/* device status bits (hs_get_status) */
#define HS_STATUS_RANGE 1u    /* a selection was >= context_len */
#define HS_STATUS_DUP 2u      /* a position appeared twice in one request's row */
#define HS_STATUS_STEP_LIMIT 4u /* a request reached 2^31-1 calls; the call was skipped */
#define HS_STATUS_TIMEOUT 8u    /* a device wait ran past the wait limit and gave up (see
                                   hs_set_wait_limit); the call's rows may be missing: hs_reset */

/* flags (hs_set_flags) */
#define HS_FLAG_NO_COPY 1u /* do all bookkeeping but skip the host->device row fetch */
/* Fault injection for tests, never for production: with it, hs_resolve's resolution
 * publishes nothing, so its overlapped fetch grid (contexts with num_requests <= the
 * SM count) waits for flags that are never raised, and hs_attend's producers withhold
 * their first fill, so its MMA issuer waits for a barrier that never completes. Every
 * such wait runs out after the wait limit: the kernels set HS_STATUS_TIMEOUT and
 * return, the context stays usable, and its cache contents are undefined until
 * hs_reset. A fetch that would not wait is not launched at all under this flag. */
#define HS_FLAG_TEST_STALL 2u

/*
 * hs_create -- one layer's cache for num_requests requests (paper abstract: full KV
 * history per request in host memory, a small fixed-size GPU cache per request).
 *   num_requests  R > 0 requests
 *   context_len   C > 0 positions of history per request (tokens, or pages)
 *   slots         S > 0 device slots per request (the GPU cache size)
 *   entry_bytes   E > 0 bytes per KV entry; a multiple of 16
 * Uses the calling thread's current CUDA device. Allocates everything up front
 * (R*C*E bytes of pinned host memory, R*S*E bytes of HBM, 4*R*(C+7S) + 268*R bytes of
 * tables, miss lists, flags and staging); hs_resolve allocates nothing. Returns NULL on failure (HS_ERR_INVALID,
 * HS_ERR_LIMIT, HS_ERR_NOMEM or HS_ERR_CUDA described by hs_last_error()). The caller
 * owns the handle and releases it with hs_destroy.
 */
hs_ctx* hs_create(int num_requests, int context_len, int slots, int entry_bytes);

/*
 * hs_create_with_host -- hs_create over a host store the caller owns and lends: the
 * caller keeps it alive (and does not free it) until hs_destroy returns. The store is
 * [R][C] rows host_stride bytes apart (a multiple of 16, >= entry_bytes), 16-byte
 * aligned, and must be pinned and mapped (cudaHostAlloc with cudaHostAllocMapped, or
 * cudaHostRegister with cudaHostRegisterMapped). Several contexts may share one store
 * (for example the layers of one model, or a pool sized by the deployment's
 * host-to-device ratio); the library only reads it. Same errors as hs_create.
 */
hs_ctx* hs_create_with_host(int num_requests, int context_len, int slots, int entry_bytes,
                            uint8_t* host_kv, size_t host_stride);

/*
 * hs_resolve -- the fused per-layer swap-in resolution (paper abstract: hit
 * detection, LRU replacement and host-to-device fetches for each layer's selections;
 * blog commentary section three: the same step updates the page table).
 *   stream        stream to enqueue on; the call is enqueue-only (no host sync, no
 *                 allocation), has a fixed launch shape and can be captured in a
 *                 CUDA graph; replays advance the per-request step counters
 *   selections    device int32 [B][k], row-major: request b's selected positions
 *   B             must equal num_requests
 *   k             0 < k <= slots
 *   out_slots     device int32 [B][k]: out_slots[b][j] is the slot now holding
 *                 selections[b][j] (-1 for padding or out-of-range); the entry's
 *                 bytes are at hs_device_kv() + ((size_t)b * S + slot) * E
 *   miss_counts   device int32 [B]: distinct missed positions of request b
 * The caller owns selections/out_slots/miss_counts and keeps them alive until the
 * enqueued work completes. The call's first kernel is a programmatic dependent of the
 * kernel before it on the stream and reads `selections` before waiting for that kernel:
 * a kernel that writes the selections and uses programmatic dependent launch itself
 * must signal completion to its dependents only after writing them (kernels that do not
 * use it have finished before this call starts). Returns HS_OK, HS_ERR_INVALID (nothing
 * enqueued) or HS_ERR_CUDA (a launch failed).
 */
int hs_resolve(hs_ctx* ctx, hs_stream_t stream, const int32_t* selections, int B, int k,
               int32_t* out_slots, int32_t* miss_counts);

/*
 * hs_resolve_host -- hs_resolve with HOST buffers; returns after the results are in
 * them (it waits for the stream). A page-locked buffer (cudaHostAlloc, cudaMallocHost,
 * or cudaHostRegister'ed and mapped; 4-byte aligned) is read or written by the kernels
 * in place over the host link, with no copy; any other host buffer (pageable memory) is
 * staged through device buffers preallocated by hs_create, with one copy each way. The
 * three buffers are classified independently. Same arguments and errors as hs_resolve.
 */
int hs_resolve_host(hs_ctx* ctx, hs_stream_t stream, const int32_t* selections_host, int B, int k,
                    int32_t* out_slots_host, int32_t* miss_counts_host);

/*
 * hs_resolve_profiled -- hs_resolve that records ev[0] before the resolution kernel,
 * ev[1] between it and the fetch kernel and ev[2] after the fetch (per-kernel timing
 * with events on the launching stream). The two kernels then run one after the other
 * instead of overlapping. ev entries must be valid events created on the context's
 * device. Results are identical to hs_resolve.
 */
int hs_resolve_profiled(hs_ctx* ctx, hs_stream_t stream, const int32_t* selections, int B, int k,
                        int32_t* out_slots, int32_t* miss_counts, hs_event_t ev[3]);

/*
 * hs_append -- decode-time append of new KV entries (blog commentary, opening: the KV
 * that does not need to stay on the GPU is offloaded to host memory; paper abstract:
 * each request's full KV history lives in host memory). Enqueues on `stream` a kernel
 * that writes kv[b] (device, [B][entry_bytes], 16-byte aligned) into the host store at
 * position positions[b] of request b (device int32 [B]; negative = no new entry for
 * that request) -- the writes cross the host link from the GPU -- and, when that
 * position is resident in a slot (a rewrite), into the slot as well, so the cache stays
 * exact. The replacement state does not change: to make a new entry resident, select it
 * in the next hs_resolve (or resolve it on its own). A position >= context_len sets
 * HS_STATUS_RANGE and is skipped. B must equal num_requests (at most 65535). Stream
 * ordered with hs_resolve on the same context. Returns HS_OK, HS_ERR_INVALID,
 * HS_ERR_LIMIT or HS_ERR_CUDA.
 */
int hs_append(hs_ctx* ctx, hs_stream_t stream, const uint8_t* kv, const int32_t* positions, int B);

/*
 * hs_attend -- the layer's consumer: sparse attention of every request over the slots
 * its selections resolved to (blog commentary, section two: a resident entry takes part
 * in the computation directly; paper abstract: only placement changes, so outputs are
 * unchanged). For the 656-byte entries of the DeepSeek sparse-attention family (the
 * context's entry_bytes must be 656): bytes [0,512) are E4M3 codes of the latent vector,
 * [512,528) four fp32 scales (scale g for codes 128g..128g+127), [528,656) 64 bf16 rotary
 * values. Key K_j = (latent_j * scale, rope_j) in R^576, value V_j = latent_j * scale in
 * R^512; for head h and the selections j with out_slots[b][j] >= 0:
 *   s_hj = sm_scale * <q_h, K_j>,  o[b][h] = sum_j softmax_j(s_h) V_j,  lse[b][h] = ln sum_j exp(s_hj).
 * A head with no valid selection gets o = 0 and lse = -inf.
 *   q          device bf16 [B][H][576], 16-byte aligned
 *   out_slots  device int32 [B][k] as written by hs_resolve (negative = not valid)
 *   o, lse     device fp32 [B][H][512] (16-byte aligned) and [B][H], overwritten
 *   workspace  device scratch of hs_attend_workspace() bytes (may be NULL when that is 0)
 * The latent codes are decoded to bf16 (code * scale rounded to nearest even), the
 * products run on the tensor cores with fp32 accumulation, and the softmax weights are
 * rounded to bf16 before the value product. B must equal num_requests, 1 <= H <= 128,
 * k >= 1. Enqueue-only: no allocation, no host synchronisation, graph-capturable. A
 * stalled pipeline sets HS_STATUS_TIMEOUT. Returns HS_OK, HS_ERR_INVALID or HS_ERR_CUDA.
 */
int hs_attend(hs_ctx* ctx, hs_stream_t stream, const void* q, int B, int H, const int32_t* out_slots, int k,
              float sm_scale, float* o, float* lse, void* workspace, size_t workspace_bytes);

/* hs_attend_workspace -- *bytes = the workspace hs_attend needs for (B, H, k) on this
 * context's device (0 when a request's keys fit one pass). Returns HS_OK or HS_ERR_INVALID. */
int hs_attend_workspace(hs_ctx* ctx, int B, int H, int k, size_t* bytes);

/*
 * hs_checksum_rows -- a stand-in for the sparse-attention consumer of a layer (blog
 * commentary, section two: a resident entry takes part in the computation directly).
 * Enqueues on `stream` a kernel that reads the k rows each request resolved to, through
 * out_slots (device int32 [B][k] from hs_resolve; negative slots are skipped), and
 * writes sums[b] = the sum modulo 2^64 of their 8-byte little-endian words (device
 * uint64 [B], overwritten). Used to measure the overlap of layer l+1's resolution with
 * layer l's consumer (paper abstract: exact layer-wise prefetching) and to check the
 * consumer's view against the host rows. B must equal num_requests (at most 65535),
 * 0 < k <= slots. Returns HS_OK, HS_ERR_INVALID, HS_ERR_LIMIT or HS_ERR_CUDA.
 */
int hs_checksum_rows(hs_ctx* ctx, hs_stream_t stream, const int32_t* out_slots, int B, int k,
                     uint64_t* sums);

/* hs_destroy -- synchronizes the device and frees everything; NULL is a no-op. */
void hs_destroy(hs_ctx* ctx);

/*
 * hs_reset -- enqueue a reset of all state to empty on `stream` (page table, slot
 * tokens and last use to -1, steps to 0, device buffer to zero, status cleared). The
 * host KV store is left as it is.
 */
int hs_reset(hs_ctx* ctx, hs_stream_t stream);

/* Host KV store: host pointer (also valid on the device through unified addressing)
 * to [R][C] rows of hs_host_stride() bytes. The caller writes the history here before
 * resolving; the library only reads it. */
uint8_t* hs_host_kv(hs_ctx* ctx);
size_t hs_host_stride(hs_ctx* ctx);

/* Device pointers to the state, for consumers and tests (layouts above). The device
 * buffer is read by the sparse-attention consumer; the tables should be treated as
 * read-only by callers. */
uint8_t* hs_device_kv(hs_ctx* ctx);
int32_t* hs_page_table(hs_ctx* ctx);
int32_t* hs_slot_token(hs_ctx* ctx);
int32_t* hs_last_use(hs_ctx* ctx);
int32_t* hs_step(hs_ctx* ctx);

/* hs_get_status -- synchronizes the device, then stores the OR of HS_STATUS_* bits
 * raised since the last hs_clear_status / hs_reset into *bits. */
int hs_get_status(hs_ctx* ctx, uint32_t* bits);
int hs_clear_status(hs_ctx* ctx);

/* hs_set_flags -- HS_FLAG_* bits for later calls (0 restores the default). */
int hs_set_flags(hs_ctx* ctx, unsigned flags);

/*
 * hs_set_wait_limit -- time limit, in nanoseconds of the GPU's global timer, of the
 * device waits of the kernels enqueued after it returns (hs_resolve's fetch grid waits
 * for its resolution's per-request flags; hs_attend's roles wait on shared-memory
 * barriers). A CTA's waits give up once it has run that long since it started; the
 * kernel then sets HS_STATUS_TIMEOUT and returns instead of spinning, so no lost
 * hand-off can hold the GPU. Default 20 ms (a healthy wait lasts microseconds); range
 * [1 us, 10 s]. Calls captured into a CUDA graph keep the limit they were captured
 * with. Not a timeout of the call as a whole: drains of in-flight copies after an
 * expiry take at most one more limit. Returns HS_OK or HS_ERR_INVALID.
 */
int hs_set_wait_limit(hs_ctx* ctx, uint64_t ns);

/* replacement policies (hs_set_policy) */
#define HS_POLICY_LRU 0    /* the method's: victims are the least recently used slots */
#define HS_POLICY_FIFO 1   /* victims are the slots filled longest ago; a hit does not renew */
#define HS_POLICY_RANDOM 2 /* victims are drawn at random among the slots not hit */

/*
 * hs_set_policy -- the replacement policy of the hs_resolve / hs_resolve_host /
 * hs_resolve_profiled calls enqueued after it returns (the blog commentary's Fig. 3
 * discussion: LRU against policies that do not exploit locality; the pages name none,
 * so the two plainest are offered for comparison). Everything but the choice of
 * victims is the same under every policy: hits, the ascending-position order of the
 * misses, the pairing of the r-th miss with the r-th victim, the page-table update.
 *   HS_POLICY_LRU     victims in ascending (last_use, slot); hits and fills stamp t
 *   HS_POLICY_FIFO    victims in ascending (last_use, slot), but a hit keeps its
 *                     stamp, which is therefore the call that filled the slot
 *   HS_POLICY_RANDOM  victims in ascending (key, slot) among the slots not hit, where
 *                     the key of slot s at call t of request b is the high 32 bits of
 *                     SplitMix64 output number t * 2^16 + s of the generator seeded
 *                     with SplitMix64 output number b of `seed` (Steele, Lea and Flood,
 *                     2014: output n of seed x is mix(x + (n + 1) * 0x9E3779B97F4A7C15),
 *                     mix being Stafford's 13th mixer); stamps are kept as under LRU
 * The state kept so far carries over (stamps mean the last use under LRU and RANDOM
 * and the fill call under FIFO from then on). Calls captured into a CUDA graph keep
 * the policy they were captured with. hs_resolve_noalloc always uses LRU.
 * Returns HS_OK or HS_ERR_INVALID (unknown policy).
 */
int hs_set_policy(hs_ctx* ctx, int policy, uint64_t seed);

/*
 * ---------------------------------------------------------------------------------
 * Capacity planning and the shared host pool (blog commentary, section on deployment
 * knobs: top_k, device_buffer_size and host_to_device_ratio set HiSparse's working range;
 * 2048 / 6144 / 10 for a disaggregated decode instance, a 4096 buffer with ratio 8 for a
 * colocated 8-GPU node). Host code only; nothing here touches a GPU.
 */
typedef struct {
    int top_k;                   /* selections per request, layer and step (k) */
    int device_buffer_size;      /* device slots per request and layer (S), >= top_k */
    double host_to_device_ratio; /* host pool rows / device pool rows, > 0 */
    int entry_bytes;             /* bytes of one KV entry (E) */
    int layers;                  /* layers, each with its own buffer and history */
    int64_t context_len;         /* positions of history a request reserves (C) */
    int64_t hbm_bytes;           /* device memory available to the caches */
    int64_t host_bytes;          /* pinned host memory available to the pool */
    double miss_fraction;        /* expected misses per step as a fraction of top_k, in [0, 1] */
    double link_gbs;             /* host-to-device bandwidth for the fetches (0: no estimate) */
} hs_plan_params;

typedef struct {
    int64_t device_bytes_per_request; /* all layers: buffer, page table, slot tables, miss lists */
    int64_t requests_by_device;       /* requests whose device state fits hbm_bytes */
    int64_t host_pool_rows;           /* ratio x requests_by_device x S, clamped to host_bytes */
    int64_t host_pool_bytes;          /* host_pool_rows x entry_bytes x layers */
    int64_t requests_by_host;         /* requests whose context_len rows fit the pool */
    int64_t requests;                 /* admissible concurrency: the smaller of the two */
    double miss_bytes_per_step;       /* host-to-device bytes of one decode step at that concurrency */
    double link_us_per_step;          /* that traffic at link_gbs (0 when link_gbs is 0) */
} hs_plan_result;

/* hs_plan -- fills *out from *in. Returns HS_OK or HS_ERR_INVALID (a value out of range). */
int hs_plan(const hs_plan_params* in, hs_plan_result* out);

/*
 * hs_pool -- the admission side of a shared host pool of `rows` rows: a request is
 * admitted by reserving a contiguous extent for its whole history (first fit: the free
 * extent with the lowest base that is long enough), and its extent is released when it
 * finishes (merged with free neighbours). The pool only does the bookkeeping; the rows
 * themselves are a pinned, mapped store the caller allocates (see hs_create_pooled).
 *   hs_pool_create   NULL if rows <= 0 or out of memory; hs_pool_destroy frees it.
 *   hs_pool_reserve  base row of a new extent of n > 0 rows, or -1 if none is long enough
 *                    (or the bookkeeping could not allocate).
 *   hs_pool_release  frees the extent reserved at `base`: HS_OK, HS_ERR_INVALID if no
 *                    extent starts there, or HS_ERR_NOMEM (the pool is left unchanged).
 *   hs_pool_free_rows, hs_pool_largest_free   free rows in total, and in one extent.
 */
typedef struct hs_pool hs_pool;
hs_pool* hs_pool_create(int64_t rows);
void hs_pool_destroy(hs_pool* pool);
int64_t hs_pool_reserve(hs_pool* pool, int64_t n);
int hs_pool_release(hs_pool* pool, int64_t base);
int64_t hs_pool_free_rows(const hs_pool* pool);
int64_t hs_pool_largest_free(const hs_pool* pool);

/*
 * hs_create_pooled -- hs_create over a shared host pool: the caller's pinned, mapped
 * store of pool_rows rows host_stride bytes apart (16-byte aligned, stride a multiple of
 * 16 >= entry_bytes; the caller keeps it alive until hs_destroy). Request b reads its
 * position p from row base[b] + p, and only positions p < len[b] exist (others are out of
 * range: slot -1, HS_STATUS_RANGE); context_len is the longest len allowed. Initially
 * every len is 0 (nothing admitted). Returns NULL on failure, as hs_create.
 */
hs_ctx* hs_create_pooled(int num_requests, int context_len, int slots, int entry_bytes, const void* host_pool,
                         int64_t pool_rows, size_t host_stride);

/*
 * hs_set_extents -- the extents of all num_requests requests of a pooled context (host
 * arrays base[R] >= 0, len[R] in [0, context_len], base + len <= pool_rows). Every request
 * whose extent changes is a new request: its cache state (page table, slots, stamps,
 * call counter, slot contents) is emptied. Enqueued on `stream` (copies from the caller's
 * arrays, which may be reused on return); an admission-time call, not meant to be
 * captured into a CUDA graph (its copies come from pageable memory). Returns HS_OK,
 * HS_ERR_INVALID or HS_ERR_CUDA.
 */
int hs_set_extents(hs_ctx* ctx, hs_stream_t stream, const int64_t* base, const int32_t* len);

/*
 * ---------------------------------------------------------------------------------
 * 4-bit pages. A KV entry may be a page: the K and V of `tokens` consecutive tokens for
 * all KV heads (Quest-style page selection; a position is then a page number). Stored in
 * 4 bits, a page crosses the host link and takes a slot at 9/32 of its 16-bit size. The
 * calls below write tokens into such pages, read pages back, and attend over the pages
 * that a resolution left in its slots. A context that holds them has entry_bytes =
 * hs_page_bytes(). All of them are enqueue-only and graph-capturable, allocate nothing and
 * need no workspace; their device pointers belong to the calling thread's current device.
 * Their kernels are programmatic dependents of the kernel before them on the stream: they
 * may be launched while it runs, and wait for it to end before they read or write anything.
 *
 * Layout: for tile i (tokens 16 i .. 16 i + 15 of the page) and head h, the 18 * head_dim
 * bytes at (i * kv_heads + h) * 18 * head_dim hold K codes [16][head_dim / 2], K scales
 * [16][head_dim / 16], V codes and V scales alike. Byte c of a row of codes holds dimension
 * 2 c in its low half and 2 c + 1 in its high half; a code is a sign bit and an E2M1
 * magnitude (0, .5, 1, 1.5, 2, 3, 4, 6). A scale byte u belongs to 16 dimensions of one
 * token and is the half-precision number whose bits are u << 7. Value = code * scale, which
 * is exact in bf16 and fp16.
 * Written from a block of 16 values x with a = max |x|: the scale s nearest to a / 6 (ties
 * to the even byte, at most 10240), codes nearest to x / s (ties to the even code, at most
 * 6; a value that rounds to zero gets code 0). A block with an infinity or a NaN gets scale
 * byte 255 and reads back as NaNs; one whose largest magnitude is under 6 * 2^-18 as zeros.
 */
typedef struct {
    int tokens;   /* of a page: a multiple of 16, at most 256 */
    int kv_heads; /* 1 .. 65535 */
    int head_dim; /* 64, 128 or 256 */
} hs_page_shape;

/* 16-bit types of K, V, q and o */
#define HS_BF16 0
#define HS_F16 1

/* hs_page_bytes -- bytes of a page, tokens * kv_heads * head_dim * 9 / 8 (0: unsupported shape). */
size_t hs_page_bytes(const hs_page_shape* shape);

/* K and V of tokens: row (token i, head h) starts i * token_stride + h * head_stride elements
 * into the tensor; rows are contiguous and 16-byte aligned (strides multiples of 8). */
typedef struct {
    const void* k;
    const void* v;
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
} hs_token_rows;

/*
 * hs_write_tokens -- quantises n tokens into pages (device memory, or pinned memory mapped
 * on the device; 16-byte aligned): token i into token slot dest[i] = page * tokens + offset
 * (device int64 [n]; negative: the token is padding and is skipped). A slot >= num_pages *
 * tokens is skipped and sets HS_STATUS_RANGE in *status (device word, or NULL). The slots of
 * one call are distinct (two tokens sent to one slot leave a mixture). Other tokens' bytes
 * are not touched. Returns HS_OK, HS_ERR_INVALID or HS_ERR_CUDA.
 */
int hs_write_tokens(hs_stream_t stream, const hs_page_shape* shape, int dtype, const hs_token_rows* rows, int64_t n,
                    const int64_t* dest, uint8_t* pages, int64_t num_pages, uint32_t* status);

/*
 * hs_append_tokens -- hs_append for tokens of 4-bit pages: token i joins request
 * requests[i] (device int32 [n]; NULL: request i, and n must be num_requests) at token
 * position positions[i] (device int32 [n]; negative: skipped), which is offset position %
 * tokens of page position / tokens. It is written into the host store and, when the page is
 * resident, into its slot as well, so the cache stays exact; the replacement state does not
 * change. A page >= context_len (or the request's extent), or a request >= num_requests, is
 * skipped and sets HS_STATUS_RANGE; a negative request is skipped like a negative position.
 * Distinct (request, position) pairs only. Stream ordered with the context's other calls.
 */
int hs_append_tokens(hs_ctx* ctx, hs_stream_t stream, const hs_page_shape* shape, int dtype, const hs_token_rows* rows,
                     int64_t n, const int32_t* requests, const int32_t* positions);

/*
 * hs_read_pages -- decodes pages: for each request b < B and j < n the page in slot
 * slots[b][j] (device int32 [B][n]) of pages [B][S] (16-byte aligned, e.g. hs_device_kv())
 * becomes tokens j * tokens .. of k[b] and v[b] (device [B][n * tokens][kv_heads][head_dim],
 * contiguous, 16-byte aligned, overwritten). A negative slot reads as zeros, one >= S too,
 * setting HS_STATUS_RANGE in *status (or NULL).
 */
int hs_read_pages(hs_stream_t stream, const hs_page_shape* shape, int dtype, const uint8_t* pages, int B, int S,
                  const int32_t* slots, int n, void* k, void* v, uint32_t* status);

/*
 * hs_attend_pages -- decode attention of every request over the pages its selections
 * resolved to. Each KV head serves q_heads / kv_heads query heads. With p_j the token
 * position of key j, qpos = lengths[b] - q_tokens + t that of query token t and, for head h,
 *   s_j = sm_scale <q, K_j>;  c_j = softcap * tanh(s_j / softcap) (softcap > 0, else s_j);
 *   x_j = c_j - slopes[h] * (qpos - p_j);
 *   o = sum_j softmax_j(x) V_j,  lse = ln sum_j exp(x_j)
 * over the keys of pages with slots[b][j] >= 0 and selections[b][j] >= 0 that have p_j <=
 * qpos and, where a document mask is given, p_j >= start[b] or p_j < prefix[b]. A query that
 * sees no key gets o = 0 and lse = -inf. Keys that no query sees are not read into the
 * result, whatever their bytes hold; a page selected twice counts twice.
 * Rows of q and o are contiguous and 16-byte aligned: (b, t, head) starts
 * b * batch_stride + t * token_stride + head * head_stride elements in; rows of o that overlap
 * are refused. A score that is -inf in f32 has a weight of 0, as if unseen (a NaN in its V still shows); a NaN key
 * makes every query that sees it NaN, in o and lse. The products run on the tensor cores with
 * f32 sums; the queries enter them as halves (bf16 ones scaled by a power of two per row) and
 * the softmax weights are rounded to half for the product with V. A capped score is within
 * 2^-20 of itself, whatever the cap; biases are f32 numbers that count from the nearest key of
 * the selected pages, or from the farthest where the slope is negative, so that the keys with
 * the largest scores keep their differences; the exponentials, and lse, are formed in base 2
 * by the GPU's approximate instructions (about 2^-22 each).
 */
typedef struct {
    hs_page_shape shape;
    int dtype;               /* of q and o: HS_BF16 or HS_F16 */
    int B, S, k;             /* requests; slots and selections of each (k may be 0) */
    int q_heads;             /* a multiple of shape.kv_heads */
    int q_tokens;            /* query tokens of each request, the last of its sequence (>= 1) */
    const void* q;
    int64_t q_batch_stride, q_token_stride, q_head_stride;
    void* o;
    int64_t o_batch_stride, o_token_stride, o_head_stride;
    float* lse;              /* device [B][q_tokens][q_heads], overwritten */
    const uint8_t* pages;    /* device [B][S] pages, 16-byte aligned (hs_device_kv()) */
    const int32_t* slots;    /* device [B][k], as written by hs_resolve */
    const int32_t* selections; /* device [B][k], the page numbers resolved */
    const int32_t* lengths;  /* device [B]: tokens of the sequence, the query tokens among them */
    float sm_scale, softcap; /* finite; softcap >= 0 (0: none) */
    const float* slopes;     /* device [q_heads], or NULL */
    const int32_t* start;    /* device [B], or NULL (no document mask; prefix is then ignored) */
    const int32_t* prefix;   /* device [B], or NULL (0) */
    uint32_t* status;        /* device word, or NULL: HS_STATUS_RANGE is set in it by a slot >= S,
                                whose page is left out */
} hs_page_attention;
int hs_attend_pages(hs_stream_t stream, const hs_page_attention* args);

/*
 * ---------------------------------------------------------------------------------
 * Latent entries. The calls below make the 656-byte entries that hs_attend reads and what goes
 * before and after it: tokens written into entries with their rotary keys rotated on the way,
 * entries read back, the two products of latent attention's absorbed form, and, for prompts, the
 * attention of its expanded form. All of them are enqueue-only and graph-capturable, allocate
 * nothing and need no workspace; their device pointers belong to the calling thread's current
 * device. Their kernels are programmatic dependents of the kernel before them on the stream: they
 * may be launched while it runs, and wait for it to end before they read or write anything.
 *
 * An entry is written from a latent of 512 values and a rotary key of 64. Each 128 latent values
 * share a scale, the smallest power of two s >= 2^-126 with 448 s >= max |x|; a code is the E4M3
 * number nearest to x / s (ties to even). A block with an infinity or a NaN gets a NaN for its
 * scale and reads back as NaNs. The rotary values are rotated in f32 and rounded once to bf16.
 */
#define HS_LATENT_ENTRY_BYTES 656

/* Rotation by position p: with c_i and s_i from row p of the table the pair (a, b) becomes
 * (a c_i - b s_i, a s_i + b c_i), 0 <= i < 32. */
typedef struct {
    const float* table;       /* device [rows][64]: 32 cosines, then 32 sines, of each position */
    int64_t rows;
    const int32_t* positions; /* device [n]: the tokens' positions */
    int halves;               /* pair i is dimensions i and i + 32; 0: 2 i and 2 i + 1 */
} hs_rotation;

/* Latents and rotary keys of tokens: token i's start i * stride elements into the tensor; each is
 * contiguous and 16-byte aligned (strides multiples of 8). */
typedef struct {
    const void* latent;
    const void* rope;
    int64_t latent_stride, rope_stride;
} hs_latent_rows;

/*
 * hs_write_latents -- n tokens (dtype HS_BF16 or HS_F16) into entries (device memory, or pinned
 * memory mapped on the device; 16-byte aligned): token i into entry dest[i] (device int64 [n];
 * negative: the token is padding and is skipped). rotation: NULL for rotary keys that are stored
 * as they are. An entry >= num_entries, or a position that the table has no row for, is skipped
 * and sets HS_STATUS_RANGE in *status (device word, or NULL). The entries of one call are distinct.
 * Returns HS_OK, HS_ERR_INVALID or HS_ERR_CUDA.
 */
int hs_write_latents(hs_stream_t stream, int dtype, const hs_latent_rows* rows, int64_t n, const hs_rotation* rotation,
                     const int64_t* dest, uint8_t* entries, int64_t num_entries, uint32_t* status);

/*
 * hs_append_latents -- hs_append for tokens: token i joins request requests[i] (device int32 [n];
 * NULL: request i, and n must be num_requests) at position positions[i] (device int32 [n];
 * negative: skipped), in the host store and, when that position is resident, in its slot as well,
 * so the cache stays exact; the replacement state does not change. The context's entry_bytes must
 * be 656. rotation->positions may be NULL: the tokens are then rotated by `positions`. A position
 * >= context_len (or the request's extent), a request >= num_requests, or a position that the
 * table has no row for is skipped and sets HS_STATUS_RANGE; a negative request is skipped like a
 * negative position. Distinct (request, position) pairs only. Stream ordered with the context's
 * other calls.
 */
int hs_append_latents(hs_ctx* ctx, hs_stream_t stream, int dtype, const hs_latent_rows* rows, int64_t n,
                      const hs_rotation* rotation, const int32_t* requests, const int32_t* positions);

/*
 * hs_read_latents -- decodes entries: for each request b < B and j < n the entry in slot
 * slots[b][j] (device int32 [B][n]) of entries [B][S] (16-byte aligned, e.g. hs_device_kv())
 * becomes latent[b][j] and rope[b][j] (device [B][n][512] and [B][n][64] of `dtype`, contiguous,
 * 16-byte aligned, overwritten). A negative slot reads as zeros, one >= S too, setting
 * HS_STATUS_RANGE in *status (or NULL). A value is code * scale rounded to `dtype`, which is exact
 * in bf16 but below 2^-126 and at 2^128, the code nearest to a latent of 248 * 2^120 or more, which
 * becomes infinite; so does what is too large for fp16.
 */
int hs_read_latents(hs_stream_t stream, int dtype, const uint8_t* entries, int B, int S, const int32_t* slots, int n,
                    void* latent, void* rope, uint32_t* status);

/* Rows of n tokens and `heads` heads, each times its head's matrix: row (token, head) of x starts
 * token * x_token_stride + head * x_head_stride elements in; w, bf16, holds a matrix of 128 rows of
 * 512 for each head, w_head_stride apart, its rows w_row_stride apart (a part of one projection's
 * weights, say; positive strides). Rows are contiguous and 16-byte aligned; out is contiguous and
 * 16-byte aligned. */
typedef struct {
    const void* x;
    int64_t x_token_stride, x_head_stride;
    const void* w;
    int64_t w_head_stride, w_row_stride;
    void* out;
    int64_t n;
    int heads; /* 1 .. 65535 */
    uint32_t* status; /* hs_expand_outputs: device word, or NULL (hs_absorb_queries takes its own) */
} hs_head_product;

/*
 * hs_absorb_queries -- the queries of the absorbed form, as hs_attend takes them: of x (bf16
 * [n][heads][128 + 64]) the first 128 values become out[..][c] = sum_d x[..][d] w[head][d][c], c <
 * 512, and the last 64, rotated (rotation: NULL if they are already), out[..][512 ..] (out: bf16
 * [n][heads][576], not x; x's strides positive, n at most 65535 * 64). bf16 products, f32 sums, one
 * rounding. A token whose position is negative gets zeros for its rotary values; so does one that the table has no row
 * for, which sets HS_STATUS_RANGE in *status (or NULL). HS_STATUS_TIMEOUT: a hand-off within the kernel
 * was lost (a defect); rows are then NaN in out[..][.. 512]. Returns HS_OK, HS_ERR_INVALID, HS_ERR_LIMIT
 * or HS_ERR_CUDA.
 */
int hs_absorb_queries(hs_stream_t stream, const hs_head_product* product, const hs_rotation* rotation, uint32_t* status);

/*
 * hs_expand_outputs -- what hs_attend gives (x: f32 [n][heads][512], strides multiples of 4)
 * through the heads' value matrices: out[..][e] = sum_c x[..][c] w[head][e][c], e < 128 (out: bf16
 * [n][heads][128]). x is taken to within 2^-15 of itself (as two bf16), the sums are f32.
 * HS_STATUS_TIMEOUT in *product->status (or NULL): a hand-off within the kernel was lost (a defect);
 * rows are then NaN.
 */
int hs_expand_outputs(hs_stream_t stream, const hs_head_product* product);

/*
 * hs_attend_prompts -- attention of B prompts in the expanded form. The rows of prompt b are
 * q_starts[b] .. q_starts[b + 1] - 1 of q, o and lse, its keys k_starts[b] .. k_starts[b + 1] - 1
 * of k, k_rope and v; there may be more keys than rows (a chunk behind earlier ones) or fewer. For
 * row i of Lq and key j of Lk, s_j = sm_scale (<q[:128], k_j> + <q[128:], k_rope_j>), over j < Lk,
 * or with `causal` j <= i + Lk - Lq: o = sum_j softmax_j(s) v_j, lse = ln sum_j exp(s_j). A row
 * that sees no key gets o = 0 and lse = -inf. Keys behind a prompt's last are not read into its
 * result, whatever they hold, and rows of q outside every prompt leave o and lse as they were. (With
 * `causal`, an infinity or a NaN among a key's values reaches rows that do not see the key, with a weight
 * of 0, so as NaN: those of the same 128, from the prompt's first row on, of which the last one sees
 * the key or one of the 15 before it.) A prompt whose starts descend, or lie
 * outside the rows there are, or whose rows begin before those of an earlier prompt end (behind
 * starts that descend), is left out and sets HS_STATUS_RANGE. The products run on the tensor
 * cores in `dtype` with f32 sums; the softmax weights are rounded to it, in fp16 to within 2^-32 of
 * the row's largest at the least. Rows of every tensor are contiguous and 16-byte aligned (strides
 * multiples of 8, positive where there is more than one row); rows of o that overlap are refused.
 * HS_STATUS_TIMEOUT: a hand-off within the kernel was lost (a defect); rows may then be NaN, or
 * missing. Returns HS_OK, HS_ERR_INVALID, HS_ERR_LIMIT or HS_ERR_CUDA.
 */
typedef struct {
    int dtype;                 /* of q, k, k_rope, v and o: HS_BF16 or HS_F16 */
    int B, heads;              /* prompts; heads 1 .. 65535 */
    int causal;
    int64_t q_rows, k_rows;    /* of the tensors */
    const void* q;             /* [q_rows][heads][128 + 64], the last 64 rotated */
    int64_t q_token_stride, q_head_stride;
    const void* k;             /* [k_rows][heads][128] */
    int64_t k_token_stride, k_head_stride;
    const void* k_rope;        /* [k_rows][64], rotated; the heads share it */
    int64_t k_rope_stride;
    const void* v;             /* [k_rows][heads][128] */
    int64_t v_token_stride, v_head_stride;
    void* o;                   /* [q_rows][heads][128] */
    int64_t o_token_stride, o_head_stride;
    float* lse;                /* device [q_rows][heads], contiguous */
    const int32_t* q_starts;   /* device [B + 1] */
    const int32_t* k_starts;   /* device [B + 1] */
    float sm_scale;            /* > 0, finite */
    uint32_t* status;          /* device word, or NULL */
} hs_prompt_attention;
int hs_attend_prompts(hs_stream_t stream, const hs_prompt_attention* args);

/*
 * hs_set_latent_waits -- for the latent calls that the calling thread makes after it returns: the
 * time limit, in nanoseconds of the GPU's global timer, of each wait within their kernels, whose
 * roles hand tiles to one another, and (10 ms where that is more) of each drain of what is still in
 * flight once a wait has run out; default 1 s, range [1 us, 10 s]. (hs_set_wait_limit's is for a CTA as a whole; one of
 * hs_attend_prompts may work for seconds, on one tile after another; while it does, or searches the
 * prompts for its next, those that wait for it do not run out.) flags: 0, or
 * HS_FLAG_TEST_STALL (tests): the kernel's first copy is announced and never made, so that the waits
 * for it run out. Calls captured into a graph keep what they were captured with. Returns HS_OK or
 * HS_ERR_INVALID.
 */
int hs_set_latent_waits(uint64_t ns, unsigned flags);

/* hs_status_word -- the context's device status word, for the calls above. */
uint32_t* hs_status_word(hs_ctx* ctx);

/* hs_device -- the CUDA device the context was created on (-1: null context). */
int hs_device(hs_ctx* ctx);

/* Number of kernels one hs_resolve call enqueues under the current flags. */
int hs_kernels_per_call(hs_ctx* ctx);

/* Description of the calling thread's last failure ("" if none). */
const char* hs_last_error(void);

/*
 * hs_resolve_noalloc -- the same resolution as hs_resolve for callers that cannot
 * allocate device memory. The paper has no counterpart: it is a packaging of the
 * same step. Engines that own all GPU memory through their own pool allocator, and
 * code that sets itself up while a stream is being captured into a CUDA graph, cannot
 * call cudaMalloc, so they cannot use hs_create. Here the caller passes every buffer,
 * laid out as for a context (R = num_requests, C = context_len, S = slots,
 * E = entry_bytes):
 *   host_kv       device-visible address of the host store, [R][C] rows host_stride
 *                 bytes apart (memory from cudaHostAlloc can be passed as is under
 *                 unified addressing); 16-byte aligned, host_stride a multiple of 16
 *   device_kv     [R][S][E] bytes, 16-byte aligned
 *   page_table    int32 [R][C]; slot_token, last_use int32 [R][S]; step int32 [R]:
 *                 the caller initialises them to -1, -1, -1 and 0 for an empty cache
 *   selections, k, out_slots, miss_counts   as for hs_resolve (B = num_requests)
 *   status        device uint32 that collects HS_STATUS_* bits, or NULL
 * It allocates nothing and calls no allocating routine. Its two kernels run one after
 * the other (hs_resolve overlaps them). The miss list the two kernels
 * share lives in a fixed file-scope device array of HS_NOALLOC_SCRATCH_BYTES bytes,
 * which every GPU that loads this library keeps until the process exits; a call needs
 * about 8*R*S + 260*R + 4*G bytes of it, G = the GPU's SM count (up to 64 more for
 * alignment) and larger sizes fail with
 * HS_ERR_LIMIT before anything is enqueued. Every call on a device shares that device's copy of the array, so calls
 * whose work overlaps on the GPU (on two streams, say) race: serialise them. The array
 * keeps the last call's contents, which the next call continues from: besides the
 * lists every call rewrites, it holds per-request flags and counters; it starts zeroed at
 * load, which is a valid state, and needs no clearing between calls. The first call on a
 * device does a one-time set-up with that device current (it looks up the array's
 * device address and sets kernel attributes): make that first call before any stream
 * capture. Returns HS_OK or HS_ERR_* (hs_last_error() describes it).
 */
#define HS_NOALLOC_SCRATCH_BYTES (2u * 1024u * 1024u)
int hs_resolve_noalloc(hs_stream_t stream, int num_requests, int context_len, int slots,
                       int entry_bytes, const uint8_t* host_kv, size_t host_stride, uint8_t* device_kv,
                       int32_t* page_table, int32_t* slot_token, int32_t* last_use, int32_t* step,
                       const int32_t* selections, int k, int32_t* out_slots, int32_t* miss_counts,
                       uint32_t* status);

#ifdef __cplusplus
}
#endif

#endif /* HS_H_ */
