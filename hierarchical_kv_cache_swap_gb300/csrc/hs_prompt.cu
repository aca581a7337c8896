// hs_prompt.cu -- attention of prompts, latent attention's expanded form: every head has keys of its
// own, 128 values expanded from the latent and the token's 64 rotary ones, which all heads share, and
// values of 128. For query row i of a prompt of Lq rows and Lk keys,
//   s_j = scale (<q_i[:128], k_j> + <q_i[128:], k_rope_j>),  o_i = sum_j softmax_j(s) v_j,  lse_i = ln sum_j exp(s_j)
// over j < Lk, or j <= i + Lk - Lq (causal): 640 operations a (query, key, head) against a few bytes,
// so the tensor cores bound it (tcgen05, bf16 or fp16 operands, f32 sums).
//
// An item is 256 rows of one head, two tiles of 128 that share every key tile of 128; a CTA walks its
// keys once, with a running maximum and sum for each row, and then takes another item from the launch
// control (a CTA of the grid that has not begun), which the roles enter one by one: the next item's keys
// and scores come while the last one's softmax and stores run. The roles:
//   * one warp looks up which rows and keys an item has;
//   * one thread copies keys, rotary keys and values through tensor maps into a ring of eight 16 KB
//     chunks (a key tile is three chunks of 64 dimensions, the rotary one read straight from the shared
//     tensor; its values are two chunks of 64 keys), each freed as soon as both row tiles have used it;
//   * one thread a row tile issues the products: S = Q K^T (128 x 128 in tensor memory, 12 instructions
//     of 16 dimensions) and O += P V (P from tensor memory, where it lies over the scores it came from).
//     The two take turns, so that while one tile's softmax runs the other's products do;
//   * four warps a row tile hold a row a thread: no value crosses lanes. The maximum m of a row moves
//     only when a tile's exceeds it by more than 8 (log2), and O is then rescaled in tensor memory; P =
//     2^(x - m) stays below 2^8 and is rounded to the operands' type for the product (2^-8 or 2^-11 of
//     each weight at most, as the queries and keys have been; fp16, held at 2^7 times P, has no better than
//     2^-32 of the kept maximum for weights below 2^-21 of it), the sum is of the unrounded f32 values. P
//     goes to the products by halves of its keys.
// Keys past a prompt's end that a tile reads (the next prompt's, or zeros behind the tensor) are masked
// in S, and their values zeroed in shared memory, whatever they hold.
//
// A key tile costs the tensor core 2560 cycles (64 an instruction). Measured on one GB300: 16384 rows of
// 16 heads, causal, 743 us = 1.85 PFLOP/s, 96 % of what a library product reaches in a burst (in a run of
// seconds the card's power limit holds both lower); 512 rows over 16384 keys of 64 heads 219 us, on the 128
// SMs that its items fill; a lone item 3500 cycles a key tile: the two turns, each 1280 cycles of products
// and about 450 of waits. Short items (64 prompts of 100 tokens, 16 heads: 32 us) cost about 7500
// cycles each, of which code that has left the instruction cache is a good part. What brought it
// there (us at 16384 rows unless said): one issuing warp that runs as a whole instead of a lone lane of a
// divergent branch, and registers moved to the softmax, 1484 -> 941; heads in groups, long tiles first, 876; an
// issuing warp a tile, in turns, 830; items from the launch control 813; tries of a wait without a hint
// of how long 788; issuing on one elected lane, without votes, 743.
//
// Every wait is bounded (hs_tc.h): on expiry the CTA records HS_STATUS_TIMEOUT, writes NaN rows, waits
// for its copies and products in flight and frees its tensor memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hs_latent.h"
#include "hs_launch.h"
#include "hs_once.h"
#include "hs_tc.h"

namespace hs {
namespace {

constexpr int kRows = 128;                      // of a row tile (the MMAs' M)
constexpr int kTileRows = 2 * kRows;            // of a CTA
constexpr int kKeys = 128;                      // of a key tile
constexpr int kQDims = kHeadDim + kRope;        // 192
constexpr uint32_t kChunk = 16384;              // 128 rows x 64 dimensions, or (V) 64 keys x 128
constexpr int kSlots = 8;                       // of the ring
constexpr int kKChunks = kQDims / 64, kVChunks = kKeys / 64, kTileChunks = kKChunks + kVChunks;
// What of a key tile lands together: the first chunk of keys, the two others, each chunk of values.
enum { kKeys0, kKeys12, kValues0, kValues1, kParts };
constexpr uint32_t kQBytes = 2 * kKChunks * kChunk;
constexpr int kSoftWarps = 8, kMmaWarp = kSoftWarps /* and the next, one for each row tile */, kCopyWarp = kMmaWarp + 2,
              kItemWarp = kCopyWarp + 1;
// Three warpgroups, launched with kLaunchRegs registers a thread; the two softmax ones take what the
// third, of the issuing threads, gives up: a row of scores stays in registers.
constexpr int kThreads = 384, kLaunchRegs = 168, kSoftRegs = 216, kIssueRegs = 72;
static_assert(2 * kSoftRegs + kIssueRegs <= 3 * kLaunchRegs, "the split stays within what the block has");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;      // row tile w: scores (P over their first half) at + 128 w
constexpr float kRescaleLog2 = 8.f;
// P is held at 2^lift times the weights: fp16 has its smallest numbers at 2^-24, so that it would lose what
// weights below that add up to (16383 of 2^-25.5 are 2^-11.5); 2^(7 + 8) is still half of its largest.
template <bool BF16>
constexpr float kLiftLog2 = BF16 ? 0.f : 7.f;

constexpr int kItems = 4;  // that may be known ahead

// What a CTA works on: 256 rows of a prompt for one head.
struct Item {
    int64_t q0, k0;  // the prompt's first row and first key
    int lq, lk;      // its rows and keys; lq = 0: there is no further item
    int row0, h;
};

struct Smem {  // beyond Q and the ring
    __align__(16) uint32_t answer[4];                    // of the launch control
    uint64_t answered, wanted;                           // an answer is there; the next item is wanted
    uint64_t item_full[kItems], item_free[kItems];
    uint64_t full[2][kParts], free[kSlots];              // full: by the parity of the key tile
    uint64_t q_full[2], q_free[2], s_full[2], p_full[2][2], o_full[2], turn[2], drain[2];  // by row tile; P by halves of the keys
    Item item[kItems];
    uint32_t tmem;
    volatile int abort;
    volatile uint32_t beat[2];                           // counts the look-up's steps, and the copies': the waits for
                                                         // an item, and for one to be wanted, may be long
};
constexpr uint32_t kSmemBytes = 1024 + kQBytes + kSlots * kChunk + sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "what a CTA may have");

// The CTAs' order: groups of `heads` heads; within one the prompts' tiles, those with the most keys
// first, and for each tile the heads. The long tiles of all heads of a group so start before its short
// ones, which then fill the SMs that finish early, while the CTAs that run at the same time share the
// keys and values of a few heads in L2.
struct Order {
    uint32_t heads, per_group;  // per_group: heads * tiles
    bool wide;                  // rows of o are 32-byte aligned
};

struct Maps {
    CUtensorMap q, k, r, v;  // as an array of four, too
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// Two values at a time: x * a + b, x + y.
__device__ __forceinline__ float2 fma2(float2 x, float a, float b) {
    float2 y;
    asm("{ .reg .b64 x, a, b, d; mov.b64 x, {%2, %3}; mov.b64 a, {%4, %4}; mov.b64 b, {%5, %5}; fma.rn.f32x2 d, x, a, b; mov.b64 {%0, %1}, d; }"
        : "=f"(y.x), "=f"(y.y) : "f"(x.x), "f"(x.y), "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("{ .reg .b64 x, y, d; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 d, x, y; mov.b64 {%0, %1}, d; }"
        : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

// Finds the prompt and the tile of it that the `at`-th of the prompts' tiles is, by one warp: 32
// prompts at a time, their tiles counted and added up over the lanes. A prompt whose bounds are not in
// order, or not within the rows there are, has no tiles, nor has one whose rows begin before the end of an
// earlier one's (behind starts that descend): no row has two writers, and the tiles are never more than
// the grid's. False: there are not so many; else *found is true for the lane whose *item is filled in.
// The search goes on from where the last one ended.
struct Search {
    int from;        // a number of prompts, a multiple of 32, that have
    int64_t before;  // so many tiles, no more than the last one looked for,
    int end;         // and this as the largest end of those whose bounds are in order
};
__device__ bool find_tile(const PromptAttention& A, int at, Search& done, Item* item, bool* found, volatile uint32_t* beat) {
    const int lane = threadIdx.x & 31;
    for (; done.from < A.B; done.from += 32) {
        if (lane == 0) beat[0] = beat[0] + 1;
        const int b = done.from + lane;
        int64_t q0 = 0, q1 = 0, k0 = 0, k1 = 0;
        bool bad = false;
        if (b < A.B) {
            q0 = A.q_starts[b], q1 = A.q_starts[b + 1];
            k0 = A.k_starts[b], k1 = A.k_starts[b + 1];
            bad = q0 < 0 || q1 < q0 || q1 > A.q_rows || k0 < 0 || k1 < k0 || k1 > A.k_rows;
        }
        int end = bad ? 0 : (int)q1;  // the largest of the lanes' so far
#pragma unroll
        for (int d = 1; d < 32; d *= 2) end = max(end, __shfl_up_sync(0xffffffffu, end, d));  // (a lane's own where there is none)
        int ahead = __shfl_up_sync(0xffffffffu, end, 1);
        ahead = lane > 0 ? max(ahead, done.end) : done.end;
        bad = bad || (b < A.B && q0 < ahead);
        if (bad) {
            if (A.status) atomicOr(A.status, 1u /* HS_STATUS_RANGE */);
            q1 = q0 = k1 = k0 = 0;
        }
        const int tiles = (int)((q1 - q0 + kTileRows - 1) / kTileRows);
        int upto = tiles;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        const bool mine = at >= done.before + upto - tiles && at < done.before + upto;
        *found = mine;
        if (mine) {
            item->q0 = q0;
            item->k0 = k0;
            item->lq = (int)(q1 - q0);
            item->lk = (int)(k1 - k0);
            item->row0 = (int)(done.before + upto - 1 - at) * kTileRows;  // the last rows, which see the most keys, first
        }
        if (__any_sync(0xffffffffu, mine)) return true;
        done.before += __shfl_sync(0xffffffffu, upto, 31);
        done.end = max(done.end, __shfl_sync(0xffffffffu, end, 31));
    }
    return false;
}

// The keys that some row of an item's row tile w sees, of which its last row sees all: row i sees the keys
// below i + 1 + lk - lq (causal), or all. And the key tiles they are in.
__device__ __forceinline__ int keys_seen(const Item& it, int w, int causal) {
    const int first = it.row0 + w * kRows;
    if (first >= it.lq) return 0;
    const int last = min(first + kRows, it.lq);
    return causal ? min(max(last - it.lq + it.lk, 0), it.lk) : it.lk;
}
__device__ __forceinline__ int key_tiles(const Item& it, int w, int causal) { return (keys_seen(it, w, causal) + kKeys - 1) / kKeys; }

// Asks for the index of a CTA of this grid that has not begun, which then never will: its work is this
// CTA's. The answer lands at `to`, counted on `bar`.
__device__ __forceinline__ void ask_for_block(uint32_t* to, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(su32(to)), "r"(su32(bar)) : "memory");
}
// Whether there was one, and its index.
__device__ __forceinline__ bool block_given(const uint32_t* from, uint32_t* index) {
    uint32_t ok, x;
    asm volatile("{ .reg .pred p; .reg .b128 r; ld.shared.b128 r, [%2]; clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;"
                 " selp.u32 %0, 1, 0, p; mov.u32 %1, 0; @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r; }"
                 : "=r"(ok), "=r"(x) : "r"(su32(from)) : "memory");
    *index = x;
    return ok != 0;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const PromptAttention A, const Order order, const __grid_constant__ Maps maps) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = base + kQBytes;
    Smem* sm = reinterpret_cast<Smem*>(ring + kSlots * kChunk);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    tma_prefetch_map(&maps.q + (tid & 3));

    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
        bar_init(&sm->answered, 1);
        bar_init(&sm->wanted, 1);
        for (int i = 0; i < kItems; ++i) {
            bar_init(&sm->item_full[i], 1);
            bar_init(&sm->item_free[i], 3 + kSoftWarps);
        }
        for (int i = 0; i < kSlots; ++i) bar_init(&sm->free[i], 2);
        for (int i = 0; i < 2 * kParts; ++i) bar_init(&sm->full[0][i], 1);
        for (int w = 0; w < 2; ++w) {
            bar_init(&sm->q_full[w], 1);
            bar_init(&sm->q_free[w], 1);
            bar_init(&sm->s_full[w], 1);
            bar_init(&sm->p_full[w][0], kRows);
            bar_init(&sm->p_full[w][1], kRows);
            bar_init(&sm->o_full[w], 1);
            bar_init(&sm->turn[w], 1);
            bar_init(&sm->drain[w], 1);
        }
        sm->abort = 0;
        sm->beat[0] = sm->beat[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc<kTmemCols>(&sm->tmem);
    fence_before();
    __syncthreads();
    fence_after();
    constexpr uint32_t tmem = 0;  // all the columns there are: the allocation can only begin at the first

    // Every role walks the same items and counts them (k), the key tiles of those before (t0) and, where it
    // needs them, a row tile's own (c0): the barriers' phases go on from item to item.
    if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        bool ok = true;
        auto wait = [&](uint64_t* b, int parity) { ok = __all_sync(0xffffffffu, ok && bar_wait(b, parity & 1, &sm->abort, A.waits.ns)); };
        if (warp == kItemWarp) {
            // ------------------------------------------------------------ items
            uint32_t index = blockIdx.x, last = 0;
            Search done{0, 0, 0};
            for (int k = 0, asked = 0;;) {
                const uint32_t group = index / order.per_group, in = index - group * order.per_group;
                const uint32_t heads = min(order.heads, A.H - group * order.heads);
                Item it;
                bool found;
                if (group != last || (int64_t)(in / heads) < done.before) done = Search{0, 0, 0};  // the prompts from the first again
                last = group;
                if (find_tile(A, (int)(in / heads), done, &it, &found, sm->beat)) {
                    if (k >= kItems) wait(&sm->item_free[k % kItems], k / kItems - 1);
                    if (!ok) break;
                    if (found) {
                        it.h = (int)(group * order.heads + in % heads);
                        sm->item[k % kItems] = it;
                        bar_arrive(&sm->item_full[k % kItems]);
                    }
                    __syncwarp();
                    ok = __all_sync(0xffffffffu, ok && bar_wait_moving(&sm->wanted, k & 1, &sm->abort, A.waits.ns, sm->beat));
                    ++k;
                }
                if (!ok) break;
                if (lane == 0) {
                    sm->beat[0] = sm->beat[0] + 1;
                    fence_async_smem();
                    bar_expect_tx(&sm->answered, sizeof sm->answer);
                    ask_for_block(sm->answer, &sm->answered);
                }
                __syncwarp();
                wait(&sm->answered, asked++);
                if (!ok) {
                    bar_drain(&sm->answered, (asked - 1) & 1, A.waits.drain);  // the answer lands before the CTA's end
                    break;
                }
                const bool more = block_given(sm->answer, &index);
                __syncwarp();
                if (!more) {
                    if (k >= kItems) wait(&sm->item_free[k % kItems], k / kItems - 1);
                    if (lane == 0) {
                        sm->item[k % kItems].lq = 0;
                        bar_arrive(&sm->item_full[k % kItems]);
                    }
                    break;
                }
            }
        } else if (warp == kCopyWarp) {
            // ------------------------------------------------------------ copies (issued by one lane)
            const bool leader = elect_one();
            int t0 = 0, issued = 0, asked0 = -1, asked1 = -1;  // chunks; the last item whose queries, by row tile, are on their way
            for (int k = 0; leader; ++k) {
                auto until = [&](uint64_t* bar, int parity) { ok = ok && bar_wait(bar, parity & 1, &sm->abort, A.waits.ns); };
                ok = ok && bar_wait_moving(&sm->item_full[k % kItems], (k / kItems) & 1, &sm->abort, A.waits.ns, sm->beat);
                const Item it = sm->item[k % kItems];
                bar_arrive(&sm->item_free[k % kItems]);
                if (!ok || it.lq == 0) break;
                const int n0 = key_tiles(it, 0, A.causal), n1 = key_tiles(it, 1, A.causal), nt = max(n0, n1);
                const int q_row = (int)it.q0 + it.row0;
                const int first = t0 * kTileChunks, end = first + nt * kTileChunks;
                for (int g = first, i = 0, c = 0;; ++g) {
                    // the first keys have room before the queries do, whose place the item before still reads
                    if (g == first + (nt > 0 ? kKChunks : 0)) {
#pragma unroll 1
                        for (int w = 0; w < 2; ++w) {
                            if (k > 0) until(&sm->q_free[w], k - 1);
                            if (!ok) break;
                            (w ? asked1 : asked0) = k;
                            if ((w ? n1 : n0) > 0) {
                                bar_expect_tx(&sm->q_full[w], kKChunks * kChunk);
                                tma_load_4d(su32(base) + w * kKChunks * kChunk, &maps.q, 0, q_row + w * kRows, 0, it.h, &sm->q_full[w]);
                            } else {
                                bar_arrive(&sm->q_full[w]);
                            }
                        }
                    }
                    // the next item is wanted: what is left of this one covers the search for it
                    if (g == max(end - 2 * kTileChunks, first)) bar_arrive(&sm->wanted);
                    if (!ok || g == end) break;
                    const int slot = g % kSlots, part = c < 2 ? c : c - 1, key = (int)it.k0 + i * kKeys;
                    if (g >= kSlots) until(&sm->free[slot], g / kSlots - 1);
                    if (!ok) break;
                    issued = g + 1;
                    sm->beat[1] = issued;
                    uint64_t* const full = &sm->full[(t0 + i) & 1][part];
                    if (c != 2) bar_expect_tx(full, part == kKeys12 ? 2 * kChunk : kChunk);
                    const uint32_t to = su32(ring) + slot * kChunk;
                    if (A.waits.stall && g == 0) {}  // (tests) announced, and never made
                    else if (c < kHeadDim / 64) tma_load_4d(to, &maps.k, 0, key, c, it.h, full);
                    else if (c < kKChunks) tma_load_2d(to, &maps.r, 0, key, full);
                    else tma_load_4d(to, &maps.v, 0, key + 64 * (c - kKChunks), 0, it.h, full);
                    if (++c == kTileChunks) c = 0, ++i;
                }
                t0 += nt;
                if (!ok) break;
            }
            // no copy may land after the CTA's end: the last key tiles', and the queries
            if (leader) {
                for (int t = max(issued / kTileChunks - 2, 0); t * kTileChunks < issued; ++t)
                    for (int part = 0; part < kParts; ++part)
                        if (issued > t * kTileChunks + (part < 2 ? part : part + 1)) bar_drain(&sm->full[t & 1][part], (t >> 1) & 1, A.waits.drain);
                for (int w = 0; w < 2; ++w) {
                    const int asked = w ? asked1 : asked0;
                    if (asked >= 0) bar_drain(&sm->q_full[w], asked & 1, A.waits.drain);
                }
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ a row tile's products (issued by one lane)
            constexpr uint32_t id_s = mma_idesc(BF16, kRows, kKeys, 0), id_o = mma_idesc(BF16, kRows, kHeadDim, 1);
            const int w = warp - kMmaWarp;
            const uint32_t q_at = smem_desc(su32(base), 16) + w * kKChunks * (kChunk / 16), k_at = smem_desc(su32(ring), 16),
                           v_at = smem_desc(su32(ring), kChunk / 2), s_col = tmem + kColS + 128 * w, o_col = tmem + kColO + 128 * w;
            const bool leader = elect_one();
            auto until = [&](uint64_t* bar, int parity) { ok = ok && bar_wait(bar, parity & 1, &sm->abort, A.waits.ns); };
            auto landed = [&](int t, int part) { until(&sm->full[t & 1][part], t >> 1); };
            // The products of one lane; a chunk's slot is free once both tiles' that read it are done.
            auto scores = [&](int t, int from, int to) {
#pragma unroll
                for (int c = from; c < to; ++c) {
                    const int slot = (t * kTileChunks + c) % kSlots;
                    const uint32_t a = q_at + c * (kChunk / 16), b = k_at + slot * (kChunk / 16);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_ss(s_col, a + 2 * k, b + 2 * k, id_s, (c | k) ? 1u : 0u);
                    mma_commit(&sm->free[slot]);
                }
                if (to == kKChunks) mma_commit(&sm->s_full[w]);
            };
            // `keys` of the tile's are seen: the products end with the 16 that the last of them is in, and no
            // later key's value comes near the tile's rows, whatever it is.
            auto values = [&](int t, int c, int add, int keys) {
                const int slot = (t * kTileChunks + kKChunks + c) % kSlots;
                const uint32_t b = v_at + slot * (kChunk / 16);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (64 * c + 16 * k < keys) mma_ts(o_col, s_col + 32 * c + 8 * k, b + 128 * k, id_o, (c | k) ? 1u : add);
                mma_commit(&sm->free[slot]);
            };
            auto skip = [&](int t, int part) {  // a part that only the other tile reads
                landed(t, part);
                if (!ok) return;
                const int g = t * kTileChunks + (part < 2 ? part : part + 1);
                bar_arrive(&sm->free[g % kSlots]);
                if (part == kKeys12) bar_arrive(&sm->free[(g + 1) % kSlots]);
            };
            // The tiles take turns, each with the products of one key tile's values and of the next one's
            // scores: interleaved, both tiles' would end together and leave the tensor core idle while
            // both softmaxes run (4050 cycles a key tile instead of 3500).
            int turns = 0;
            auto take = [&] {
                if (w == 1 || turns > 0) until(&sm->turn[w], turns - (w == 0));
                ++turns;
            };
            auto give = [&] { if (ok) bar_arrive(&sm->turn[1 - w]); };
            int t0 = 0, c0 = 0;
            for (int k = 0; leader; ++k) {  // one lane alone: a vote after each wait costs more than the wait
                ok = ok && bar_wait_moving(&sm->item_full[k % kItems], (k / kItems) & 1, &sm->abort, A.waits.ns, sm->beat);
                const Item it = sm->item[k % kItems];
                bar_arrive(&sm->item_free[k % kItems]);
                if (!ok || it.lq == 0) break;
                const int n = key_tiles(it, w, A.causal), nt = max(n, key_tiles(it, 1 - w, A.causal)), seen = keys_seen(it, w, A.causal);
                // Of every item, or this warp could give the queries' place back twice before the copies
                // take it once: a wait for the first time would then see the phase after it.
                until(&sm->q_full[w], k);
                if (n == 0 && ok) bar_arrive(&sm->q_free[w]);
                if (n > 0) {
                    landed(t0, kKeys0);
                    landed(t0, kKeys12);
                }
                if (nt > 0) {
                    take();
                    fence_after();
                    if (ok && n > 0) scores(t0, 0, kKChunks);
                    give();
                    if (n == 0) skip(t0, kKeys0), skip(t0, kKeys12);
                }
                if (ok && n == 1) mma_commit(&sm->q_free[w]);
                for (int i = 0; ok && i < nt; ++i) {
                    const bool next = i + 1 < n;
                    const int t = t0 + i;
                    if (i < n) {  // what has had the time to land is waited for before the turn
                        landed(t, kValues0);
                        landed(t, kValues1);
                        if (next) landed(t + 1, kKeys0);
                        until(&sm->p_full[w][0], c0 + i);
                    }
                    take();
                    if (ok && i < n) {
                        fence_after();
                        values(t, 0, i, seen - i * kKeys);
                        until(&sm->p_full[w][1], c0 + i);
                        fence_after();
                        if (ok) values(t, 1, i, seen - i * kKeys);
                        if (ok && next) {
                            scores(t + 1, 0, 1);
                            landed(t + 1, kKeys12);
                            fence_after();
                            if (ok) scores(t + 1, 1, kKChunks);
                            if (i + 2 == n) mma_commit(&sm->q_free[w]);
                        } else if (ok) {
                            mma_commit(&sm->o_full[w]);
                        }
                    }
                    give();
                    if (i >= n) skip(t, kValues0), skip(t, kValues1);
                    if (!next && i + 1 < nt) skip(t + 1, kKeys0), skip(t + 1, kKeys12);
                }
                t0 += nt;
                c0 += n;
                if (!ok) break;
            }
            __syncwarp();
            // whatever happened, every product issued here is done before the columns are freed. (O is free for
            // an item's first values as soon as its first P is there: the same threads had read O before.)
            if (leader) mma_commit(&sm->drain[w]);
            bar_drain(&sm->drain[w], 0, A.waits.drain);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ------------------------------------------------------------ softmax, a row a thread
        const int w = warp >> 2;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, s_at = tmem + lanes + kColS + 128 * w, o_at = tmem + lanes + kColO + 128 * w;
        const float scale = A.scale * 1.4426950408889634f;
        bool ok = true;
        int t0 = 0, c0 = 0, items = 0;
        for (int k = 0;; ++k) {
            ok = __all_sync(0xffffffffu, bar_wait_moving(&sm->item_full[k % kItems], (k / kItems) & 1, &sm->abort, A.waits.ns, sm->beat));
            if (!ok) break;
            const Item& it = sm->item[k % kItems];  // until it is given back
            if (it.lq == 0) break;
            const int n = key_tiles(it, w, A.causal), nt = max(n, key_tiles(it, 1 - w, A.causal)), lk = it.lk;
            const int row = it.row0 + w * kRows + (tid & (kRows - 1));  // of the prompt
            const int seen = row < it.lq ? (A.causal ? min(max(row + 1 - it.lq + lk, 0), lk) : lk) : 0;
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < n; ++i) {
                const int here = seen - i * kKeys;  // keys of this tile that the row sees
                ok = ok && bar_wait(&sm->s_full[w], (c0 + i) & 1, &sm->abort, A.waits.ns);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                fence_after();
                uint32_t s[128];
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                const bool masked = __any_sync(0xffffffffu, here < kKeys);
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_load32(s + 32 * c, s_at + 32 * c);
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // the second half is on its way while the first is looked through
                    tmem_wait_ld();
                    if (half == 0) {
#pragma unroll
                        for (int c = 2; c < 4; ++c) tmem_load32(s + 32 * c, s_at + 32 * c);
                    }
                    if (masked) {
#pragma unroll
                        for (int c = 2 * half; c < 2 * half + 2; ++c) {
                            const int left = here - 32 * c;  // of these 32 keys
                            const uint32_t keep = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!(keep >> j & 1u)) s[32 * c + j] = __float_as_uint(-INFINITY);
                        }
                    }
#pragma unroll
                    for (int j = 64 * half; j < 64 * half + 64; j += 8)
#pragma unroll
                        for (int x = 0; x < 4; ++x) top[x] = max3(top[x], __uint_as_float(s[j + 2 * x]), __uint_as_float(s[j + 2 * x + 1]));
                }
                const float best = max3(fmaxf(top[0], top[1]), top[2], top[3]) * scale;
                const bool move = best > m + kRescaleLog2 || (m == -INFINITY && best > -INFINITY);
                if (i > 0 && __any_sync(0xffffffffu, move)) {
                    // O holds tiles 0 .. i - 1: their products ended before these scores did
                    const float f = move ? ex2(m - best) : 1.f;  // m = -inf: O is zero so far
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tmem_load32(o, o_at + 32 * c);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_store32(o_at + 32 * c, o);
                    }
                    l *= f;
                }
                if (move) m = best;
                const float from = m == -INFINITY ? 0.f : kLiftLog2<BF16> - m;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t p[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float2 x = fma2(make_float2(__uint_as_float(s[64 * c + 2 * j]), __uint_as_float(s[64 * c + 2 * j + 1])), scale, from);
                        x = make_float2(ex2(x.x), ex2(x.y));
                        sum[j & 1] = add2(sum[j & 1], x);
                        p[j] = pack<BF16>(x.x, x.y);
                    }
                    tmem_store32(s_at + 32 * c, p);
                    const int live = lk - i * kKeys - 64 * c;
                    if (live < 64) {  // values behind the prompt's end become zeros
                        // (the scores are there, so the fill before this one of the barrier is over)
                        const int t = t0 + i, first = max(live, 0);
                        ok = ok && bar_wait(&sm->full[t & 1][kValues0 + c], (t >> 1) & 1, &sm->abort, A.waits.ns);
                        uint4* at = reinterpret_cast<uint4*>(ring + (t * kTileChunks + kKChunks + c) % kSlots * kChunk);
                        for (int u = tid & (kRows - 1); ok && u < (64 - first) * 16; u += kRows)
                            at[(u & 8 ? 512 : 0) + (first + (u >> 4)) * 8 + (u & 7)] = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                        __syncwarp();  // what follows is the whole warp's
                    }
                    tmem_wait_st();
                    fence_before();
                    bar_arrive(&sm->p_full[w][c]);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            // o_full counts the items that have values: for each of them the products wait for these warps
            if (n > 0) ok = __all_sync(0xffffffffu, ok && bar_wait(&sm->o_full[w], items++ & 1, &sm->abort, A.waits.ns));
            fence_after();
            const float inv = l != 0.f ? 1.f / l : 0.f, none = __uint_as_float(0x7FC00000u);
            const int64_t to = it.q0 + row;
            const bool there = row < it.lq;
            const int h = it.h;
            __syncwarp();
            if (lane == 0) bar_arrive(&sm->item_free[k % kItems]);
            uint16_t* const out = A.o + to * A.o_token + h * A.o_head;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {  // 32 columns at a time: code that runs once for an item is kept short
                uint32_t o[32], r[16];
                if (n > 0) {
                    tmem_load32(o, o_at + 32 * c);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t both = pack<BF16>(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                    r[j] = !ok ? 0x7FFF7FFFu : l == 0.f ? 0u : both;
                }
                if (!there) continue;
                uint16_t* const at = out + 32 * c;
                if (order.wide) {
#pragma unroll
                    for (int j = 0; j < 16; j += 8)
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at + 2 * j), "r"(r[j]), "r"(r[j + 1]),
                                     "r"(r[j + 2]), "r"(r[j + 3]), "r"(r[j + 4]), "r"(r[j + 5]), "r"(r[j + 6]), "r"(r[j + 7]) : "memory");
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) reinterpret_cast<uint4*>(at)[j] = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                }
            }
            if (there)
                A.lse[to * A.H + h] = !ok ? none : l == 0.f ? -INFINITY : (m + lg2(BF16 ? l : l * 0x1p-7f)) * 0.69314718055994531f;
            t0 += nt;
            c0 += n;
            if (!ok) break;
        }
        if (!ok && lane == 0 && A.status) atomicOr(A.status, 8u /* HS_STATUS_TIMEOUT */);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        tmem_free<kTmemCols>(sm->tmem);
    }
}

bool encode_rope(CUtensorMap* map, bool bf16, const uint16_t* x, int64_t tokens, int64_t token) {
    const EncodeTiled enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t size[2] = {(cuuint64_t)kRope, (cuuint64_t)tokens}, stride[1] = {(cuuint64_t)token * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)kKeys}, step[2] = {1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<uint16_t*>(x), size, stride, box,
               step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Ready {};

}  // namespace

cudaError_t launch_attend_prompts(cudaStream_t stream, bool bf16, const PromptAttention& a) {
    if (a.B == 0 || (a.q_rows == 0 && !a.status)) return cudaSuccess;
    static PerDevice<Ready> devices;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device >= PerDevice<Ready>::kDevices) return cudaErrorInvalidDevice;
    const Ready* ready;
    e = (cudaError_t)devices.get(device, [](Ready*) {
        for (auto kernel : {prompt_kernel<true>, prompt_kernel<false>}) {
            cudaFuncAttributes at;
            cudaError_t x = cudaFuncGetAttributes(&at, kernel);
            if (x == cudaSuccess && at.numRegs < kLaunchRegs) x = cudaErrorInvalidKernelImage;  // the warps' split of them would not add up
            if (x == cudaSuccess) x = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
            if (x != cudaSuccess) return (int)x;
        }
        return 0;
    }, &ready);
    if (e != cudaSuccess) return e;
    Maps maps;
    // Without keys, or rows, no copy is made of them: their maps then are of one row at some aligned address.
    const bool rows = a.q_rows > 0, keys = rows && a.k_rows > 0;
    const uint16_t* const nothing = (const uint16_t*)((uintptr_t)a.q_starts & ~uintptr_t(15));
    const int64_t m = rows ? a.q_rows : 1, n = keys ? a.k_rows : 1;
    const int64_t q_head = rows && a.H > 1 ? a.q_head : kQDims, q_token = m > 1 ? a.q_token : kQDims;
    const int64_t k_head = keys && a.H > 1 ? a.k_head : kHeadDim, v_head = keys && a.H > 1 ? a.v_head : kHeadDim;
    const int64_t k_token = n > 1 ? a.k_token : kHeadDim, v_token = n > 1 ? a.v_token : kHeadDim;
    const int64_t r_token = n > 1 ? a.r_token : kRope;
    if (!encode_columns(&maps.q, bf16, rows ? a.q : nothing, m, kQDims / 64, a.H, q_token, q_head, kRows, kKChunks) ||
        !encode_columns(&maps.k, bf16, keys ? a.k : nothing, n, kHeadDim / 64, a.H, k_token, k_head, kKeys, 1) ||
        !encode_columns(&maps.v, bf16, keys ? a.v : nothing, n, kHeadDim / 64, a.H, v_token, v_head, 64, kHeadDim / 64) ||
        !encode_rope(&maps.r, bf16, keys ? a.k_rope : nothing, n, r_token))
        return cudaErrorInvalidValue;
    // a CTA for every 256 rows of a prompt, at most one more than full ones for each prompt; without rows one,
    // which only looks the starts over
    const int64_t tiles = rows ? a.q_rows / kTileRows + a.B : 1;
    // as many heads to a group as keep their keys and values in 64 MB, half of L2, and at most 16
    constexpr int64_t kShared = 64 << 20;
    const int64_t fit = kShared / ((a.k_rows > 0 ? a.k_rows : 1) * 4 * kHeadDim), heads = fit < 1 ? 1 : fit < 16 ? fit : 16;
    Order order;
    order.heads = (uint32_t)(heads < a.H ? heads : a.H);
    order.per_group = (uint32_t)(order.heads * tiles);
    order.wide = (((uintptr_t)a.o | (uintptr_t)(a.o_token * 2) | (uintptr_t)(a.o_head * 2)) & 31) == 0;
    return launch_dependent(stream, dim3((unsigned)(rows ? tiles * a.H : 1)), kThreads, kSmemBytes, bf16 ? prompt_kernel<true> : prompt_kernel<false>, a, order,
                            maps);
}

}  // namespace hs
