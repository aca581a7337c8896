// hs_page_attend.cu -- decode attention over resolved 4-bit pages (format: hs_page.cu).
//
// For each request b, KV head h and the G query heads that share it, the rows r = (query
// token t, head g of the group) see the keys j of the selected pages: with d_j = qpos_t - p_j
// the distance of key position p_j from the row's own position qpos_t = length - Tq + t,
//   s_j = scale <q_r, K_j>;  c_j = cap tanh(s_j / cap) (cap > 0);  x_j = c_j - slope_r d_j;
//   o_r = sum_j softmax_j(x) V_j;  lse_r = ln sum_j exp(x_j),
// over the keys with a valid slot, p_j <= qpos_t and (p_j >= start or p_j < prefix). A row
// that sees no key gets o = 0, lse = -inf.
//
// What bounds it: each key and head costs 9/8 D bytes of HBM and 2 D multiply-adds a row, so
// up to about 16 rows the stream of pages is the floor, and the work per byte -- a conversion
// and a scaling for each pair of codes, and their instructions' issue rather than any one
// pipe -- has to stay under it. So nothing decoded goes through shared memory: a warp decodes its tile's codes
// straight into the registers in which the tensor cores (mma.sync m16n8k16, f16 operands, f32
// sums) take them. Both products are formed transposed, keys (or dimensions) along the 16
// rows of the instruction and the query rows along its 8 columns, so that a group of up to 8
// query rows costs one instruction where the other way round would pad it to 16.
//
// Work split: one CTA per (request, KV head, tile of query rows, share of the selection); a
// selection is shared by up to 8 CTAs, one thread-block cluster, when there are few requests
// and heads. Each of the CTA's warps takes 16-token tiles in turn (18 D contiguous bytes,
// copied asynchronously into the warp's own ring of stages: no barrier between warps) and
// keeps its own maxima, sums and outputs; the warps are joined through shared memory at the
// end and the CTAs of a cluster through distributed shared memory, so no workspace and no
// second kernel.
//
//   S^T = K Q^T  A: 16 keys x 16 dims. Which 4 dimensions a lane holds at a step is free as
//                long as Q's do the same: lane (g, t) = (lane / 4, lane % 4) takes dimensions
//                t D/4 + 4 i ... of keys g and g + 8 at step i, so its codes are D/8
//                contiguous bytes of a row and its scales D/64 bytes.
//   O^T = V^T P  A: 16 dims x 16 keys. Lane (g, t) needs pairs of keys (2t, 2t+1) and (2t+8,
//                2t+9) for the same dimension: it takes the same bytes of four tokens and
//                interleaves their codes before decoding them. At step i it holds dimensions
//                g D/8 + 2 i and + 1.
//   P            leaves S^T's layout (a lane has keys g, g + 8 of rows 2t, 2t + 1) for the
//                other operand's (keys 2t, 2t + 1 of row g) by a transposing register move.
//
// Decoded keys and values are exact halves (hs_page.cu). Queries become halves too: fp16 ones
// as they are, bf16 ones scaled per row by a power of two that brings the row's largest
// magnitude to [2^13, 2^14), which keeps all eight bits of every component down to 2^-27 of
// the largest; what is below is rounded by at most 2^-38 of the largest. Softmax weights are
// rounded to half (2^-11 relative, unless below 2^-14 of the largest) for the second product
// only; the sums that normalise them add the unrounded ones in f32.
//
// Measured (16-token pages, 8 heads of 128 with 8 queries each, 128 pages a request; us a
// call in a graph): 256 requests 105 (5.84 TB/s, 87 % of a copy's rate), of which the copies
// alone take 91.5 and the arithmetic alone 101.5; 64 requests 33 (4.65 TB/s: 512 jobs do
// not spread evenly over 152 SMs), 1 request 5.2 and one of five tokens 3.7 (the chain of
// loads, one pair of tiles and the joins). 32 rows (four drafted tokens) over 16 requests take
// 21.7, where the products alone would take 8.5 on all SMs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <math.h>

#include "hs_once.h"
#include "hs_page.h"

namespace hs {
namespace {

constexpr int kMaxWarps = 20;
constexpr int kMaxSplit = 8;           // CTAs that share a selection: the portable cluster size
constexpr int kList = 64;              // a warp's list of live tiles (a ring; 32 are added at a time)
constexpr float kRescale = 8.f;        // a row's reference maximum moves when exceeded by 2^8
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

// A call's work split. Jobs are (request, KV head, tile of rows); a cluster of `shares` CTAs
// takes that many whole jobs while there are any and then shares one.
struct Split {
    Divisor shares, row_tiles, heads, tiles, group;  // CTAs of a cluster; ...; tiles of a page; query heads of a KV head
    int whole;             // clusters of whole jobs
    int ntiles;            // of a selection
    int groups, groups_1;  // a warp's groups of 32 tiles, of a shared job and of a whole one
};

template <int D, int NT>
struct Config {
    static constexpr int kChunk = 18 * D;           // bytes of a tile of one head
    static constexpr int kRows = 8 * NT;            // query rows of a CTA
    static constexpr int kSteps = D / 16;
    // Warps of an SM: what the registers allow (96, 128, 168 or 255 of them)
    static constexpr int kSmWarps = D == 256 ? 8 : NT == 1 ? 20 : NT * D <= 128 ? 16 : NT * D <= 256 ? 12 : 8;
    static constexpr int kStages = D == 64 ? 4 : 2;  // of two tiles
    // shared memory of a warp: its ring, over it at the end its outputs, and its list
    static constexpr int kRing = kStages * 2 * kChunk, kPart = kRows * D * 4, kListBytes = kList * 8;
    static constexpr int kSpace = (kRing > kPart ? kRing : kPart) + kListBytes;
    static int smem(int warps, int shares);
};

template <int D, int NT>
struct Fixed {  // followed by the warps' regions and, with several shares, theirs (kPart and a little)
    using C = Config<D, NT>;
    uint2 qf[NT][C::kSteps][32];              // Q as the lanes take it
    alignas(8) float qscale[C::kRows];           // of the rows: to log2 units
    alignas(8) float slope[2][C::kRows];         // [0] those from zero up, [1] those below; else 0
    int qpos[C::kRows];
    alignas(16) float2 ml[kMaxWarps][C::kRows];  // the warps' maxima and sums
    alignas(16) float2 xml[kMaxSplit][C::kRows]; // the shares'
    int2 wref[kMaxWarps], xref[kMaxSplit];       // positions that biases are relative to
};
template <int D, int NT>
int Config<D, NT>::smem(int warps, int shares) {
    return (int)((sizeof(Fixed<D, NT>) + 127) / 128 * 128) + warps * kSpace + (shares > 1 ? kPart + shares * 32 : 0);
}

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
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
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Four bytes of codes to four pairs of halves (exact).
__device__ __forceinline__ void decode_word(uint32_t w, uint32_t (&h)[4]) {
    asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b;"
        " cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t scale2(uint32_t u) { return u * 0x00800080u; }  // (s, s) of scale byte u
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Two f32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; fma.rn.f32x2 d, a, b, c;"
        " mov.b64 {%0, %1}, d; }"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2f(float2 a, float2 b) {
    float2 d;
    asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// c tanh(x / c) for two scores x in log2 units, within 2^-20 of itself at any c; to_y = 2 log2 e / c,
// so that y = x to_y has 2^y = e^(2 x / c). c - 2 c / (1 + 2^y) is off by parts of c: it serves
// from |x| = .4 c, where rounding takes at most 8 x 2^-23 of it. Below, x + x v P(v) with v = y^2
// keeps x's own precision however large c is: P is the quadratic that brings the sum nearest to
// the tanh there (least largest error, 2^-23). `far`: some score of the warp is not below; both
// forms are then made and one is selected. (24 requests with 4 x 6 heads of 64 and a cap that few
// scores come near, 14.2 us: both forms always .35 us more, and the choice left to the compiler
// another .25.)
constexpr float kNear = 0.39f;  // of the cap
__device__ __forceinline__ float2 capped(float2 x, float c, float to_y, bool far) {
    auto both = [](float a) { return make_float2(a, a); };
    const float2 y = mul2f(x, both(to_y)), v = mul2f(y, y);
    float2 p = fma2(v, both(-8.2822472e-5f), both(1.9155892e-3f));
    p = fma2(v, p, both(-0.040036008f));
    p = fma2(mul2f(x, v), p, x);
    if (!far) return p;
    auto one = [&](float y, float p) {
        const float f = fmaf(-2.f * c, rcp(1.f + ex2(y)), c);
        float r;
        asm("{ .reg .pred below; setp.lt.f32 below, %1, 0f3F93BB62; selp.f32 %0, %2, %3, below; }"  // 1.154156, .4 of the cap
            : "=f"(r) : "f"(fabsf(y)), "f"(p), "f"(f));
        return r;
    };
    return make_float2(one(y.x, p.x), one(y.y, p.y));
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN if one of them is
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 16 bytes into shared memory, asynchronously; copies are waited for by groups.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores to the place of `p` in another CTA of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(su32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void peer_store(void* p, int rank, const float4& v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(peer(p, rank)), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void peer_store(int2* p, int rank, int2 v) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(peer(p, rank)), "r"(v.x), "r"(v.y) : "memory");
}

// MOD: scores are capped or biased.
template <int D, int NT, bool MOD>
__global__ void __launch_bounds__(Config<D, NT>::kSmWarps * 32, 1) attend_pages_kernel(const PageAttention A, const Split P, bool bf16) {
    using C = Config<D, NT>;
    extern __shared__ __align__(128) uint8_t raw[];
    Fixed<D, NT>& sm = *reinterpret_cast<Fixed<D, NT>*>(raw);
    uint8_t* const space = raw + (sizeof(Fixed<D, NT>) + 127) / 128 * 128;
    const int threads = blockDim.x, warps = threads >> 5;
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known uniform, so that its loops and addresses are
    const int cluster = P.shares((int)blockIdx.x), rank = blockIdx.x - cluster * P.shares.d;
    const bool whole = cluster < P.whole;
    const int nsplit = whole ? 1 : P.shares.d, split = whole ? 0 : rank;
    const int job = whole ? cluster * (int)P.shares.d + rank : P.whole * ((int)P.shares.d - 1) + cluster;
    const int bh = P.row_tiles(job), r0 = (job - bh * (int)P.row_tiles.d) * C::kRows;
    const int b = P.heads(bh), h = bh - b * A.H;
    const int rows = A.G * A.Tq;
    uint8_t* ring = space + warp * C::kSpace;
    int2* list = reinterpret_cast<int2*>(ring + C::kSpace - C::kListBytes);
    if (nsplit > 1) cluster_arrive();  // waited for before the first store to another CTA
    // The launch may begin before the kernel ahead of it on the stream is done: nothing that
    // it reads or writes is touched before this.
    asm volatile("" ::"l"(A.slots), "l"(A.sel), "l"(A.lengths), "l"(A.q), "l"(A.pages), "r"(P.ntiles), "r"(P.tiles.m), "r"(P.group.m));
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---------------- this warp's tiles: every (nsplit * warps)-th of the selection. Lane i
    // looks up the i-th of the next 32; those that hold a visible key go on the warp's list.
    const int32_t* slots = A.slots + (size_t)b * A.k;
    const int32_t* sel = A.sel + (size_t)b * A.k;
    const int ntiles = P.ntiles, stride = nsplit * warps;
    int next = lane * stride + split * warps + warp;  // this lane's tile of the next group
    int gslot = -1, gsel = -1;                          // its page, loaded a group ahead
    auto look_up = [&]() {
        gslot = -1;
        if (next < ntiles) {
            const int j = P.tiles(next);
            gslot = load(slots + j);
            gsel = load(sel + j);
        }
    };
    look_up();
    // the request's mask: query token t sees p <= length - Tq + t and (p >= start or p < prefix)
    const int length = load(A.lengths + b);
    const int start = A.start ? load(A.start + b) : 0;
    const int prefix = A.prefix ? load(A.prefix + b) : 0;
    const int qpos0 = length - A.Tq;  // may be negative
    const uint8_t* pages = A.pages + ((size_t)b * A.S * A.tiles * A.H + h) * C::kChunk;
    const size_t unit_bytes = (size_t)A.H * C::kChunk;

    // the first of this warp's query rows (half a warp a row), on their way meanwhile
    constexpr int kQ = D / 16;  // values of a lane
    const int hl = lane & 15;
    uint32_t qw[kQ / 2];
    auto load_q = [&](int r) {
        const int row = min(r0 + r, rows - 1), tok = P.group(row), head = h * A.G + row - tok * A.G;
        const uint16_t* src = A.q + b * A.q_batch + tok * A.q_token + head * A.q_head + hl * kQ;
        if constexpr (kQ == 4) {
            const uint2 v = load(reinterpret_cast<const uint2*>(src));
            qw[0] = v.x; qw[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < kQ / 8; ++i) {
                const uint4 v = load(reinterpret_cast<const uint4*>(src) + i);
                qw[4 * i] = v.x; qw[4 * i + 1] = v.y; qw[4 * i + 2] = v.z; qw[4 * i + 3] = v.w;
            }
        }
    };
    if (2 * warp < C::kRows) load_q(2 * warp + (lane >> 4));

    int groups = whole ? P.groups_1 : P.groups;  // not yet on the list
    uint32_t fill = 0, used = 0, tail = 0;       // listed tiles copied (or on their way), consumed, listed
    int fst = 0, ust = 0;                        // the stage of the next copy and of the next wait
    auto append = [&]() {
        bool live = false;
        int2 e;
        if (gslot >= A.S && A.status) atomicOr(A.status, 1u /* HS_STATUS_RANGE */);
        if (gslot >= 0 && gslot < A.S && gsel >= 0) {
            const int tile = next - P.tiles(next) * A.tiles;
            const int64_t at = (int64_t)gsel * (A.tiles * kTile) + tile * kTile;
            if (at < length) {
                const int pos = (int)at, end = pos + (kTile - 1);
                const bool full = end <= qpos0 && (!A.start || pos >= start || end < prefix);
                live = !A.start || end >= start || pos < prefix;
                e = make_int2(gslot * A.tiles + tile, pos | (full ? 0 : 1));
            }
        }
        const uint32_t which = __ballot_sync(0xffffffffu, live);
        if (live) list[(tail + __popc(which & ((1u << lane) - 1u))) % kList] = e;
        tail += __popc(which);
        --groups;
        next = ntiles - next > 32 * stride ? next + 32 * stride : ntiles;
        look_up();
        __syncwarp();
    };
    auto top_up = [&]() {  // put the next two tiles (the last one alone) on their way, as one group
        while (tail - fill < 2 && groups > 0) append();
        const int n = min(2, (int)(tail - fill));
        if (n > 0) {
            constexpr int kParts = C::kChunk / 16;
            const int4 e = *reinterpret_cast<const int4*>(&list[fill % kList]);
            const uint8_t* from0 = pages + (size_t)e.x * unit_bytes + 16 * lane;
            const uint8_t* from1 = pages + (size_t)e.z * unit_bytes + 16 * lane - C::kChunk;
            const uint32_t to = su32(ring) + fst * (2 * C::kChunk) + 16 * lane;
#pragma unroll
            for (int i = 0; i < (2 * kParts + 31) / 32; ++i) {  // part 32 i + lane of the two tiles
                const bool first = 32 * i + 31 < kParts || (32 * i < kParts && 32 * i + lane < kParts);
                if (first) copy16(to + 512 * i, from0 + 512 * i);
                else if (n == 2 && (32 * i + 31 < 2 * kParts || 32 * i + lane < 2 * kParts)) copy16(to + 512 * i, from1 + 512 * i);
            }
        }
        copy_commit();
        fill += n;
        fst = fst + 1 == C::kStages ? 0 : fst + 1;
    };
#pragma unroll 1
    for (int i = 0; i < C::kStages; ++i) top_up();

    // ---------------- the query rows as halves, in the lanes' order
    bool below = false;  // some row's slope is below zero
    for (int r2 = 2 * warp; r2 < C::kRows; r2 += 2 * warps) {
        const int r = r2 + (lane >> 4), row = r0 + r, tok = P.group(min(row, rows - 1));
        float x[kQ], scale = 0.f, amax = 0.f;
        if (r2 != 2 * warp) load_q(r);
#pragma unroll
        for (int i = 0; i < kQ; ++i) x[i] = 0.f;
        if (row < rows) {
#pragma unroll
            for (int i = 0; i < kQ; ++i) {
                const uint32_t u = qw[i / 2] >> (16 * (i & 1)) & 0xFFFFu;
                x[i] = bf16 ? __uint_as_float(u << 16) : __half2float(__ushort_as_half((uint16_t)u));
                amax = fmaxf(amax, fabsf(x[i]));
            }
            scale = 1.f;
        }
        if (bf16) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (amax > 0.f && amax < INFINITY) {
                const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 13, -100);
                scale = __uint_as_float((uint32_t)(127 + e) << 23);
                const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int i = 0; i < kQ; ++i) x[i] *= inv;
            }
        }
        if (hl == 0) {
            sm.qscale[r] = scale * (A.scale * kLog2e);  // to log2 units
            const float slope = MOD && A.slopes && row < rows ? load(A.slopes + h * A.G + row - tok * A.G) * kLog2e : 0.f;
            below |= slope < 0.f;
            sm.slope[0][r] = slope < 0.f ? 0.f : slope;
            sm.slope[1][r] = slope < 0.f ? slope : 0.f;
            sm.qpos[r] = qpos0 + tok;
        }
        // dimension d is taken by lane d / (D/4) of the row's group at step d % (D/4) / 4
#pragma unroll
        for (int i = 0; i < kQ; i += 4)
            sm.qf[r / 8][((hl & 3) * kQ + i) / 4][(r & 7) * 4 + (hl >> 2)] = make_uint2(pack_half(x[i], x[i + 1]), pack_half(x[i + 2], x[i + 3]));
    }
    if (MOD) below = __syncthreads_or(below);
    else __syncthreads();

    float2 qs[NT];  // rows 8 n + 2 t, + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) qs[n] = *reinterpret_cast<const float2*>(&sm.qscale[8 * n + 2 * t]);
    const float cap2 = A.cap * kLog2e, to_y = 2.f / A.cap;

    // O^T: dims g D/8 + 2 i (c = 0, 1), + 1 (2, 3); rows 8 n + 2 t (c = 0, 2), + 1 (1, 3)
    float acc[C::kSteps][NT][4];
    float2 m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = make_float2(-INFINITY, -INFINITY);
        l[n] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < C::kSteps; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][n][c] = 0.f;
    }
    // A row's biases are relative to the last position of the tiles so far (x), or to the first
    // (y) where its slope is negative: the keys with the largest scores keep small biases.
    int2 ref = make_int2(0, INT_MAX);
    const bool biased = MOD && A.slopes;
    // The order of a tile's keys along the instruction: place r holds token order(r). A lane's
    // four tokens of V (places 2t, 2t + 1, + 8) then lie in both halves of the 128 bytes that
    // the shared memory banks cover, and its keys still do.
    auto order = [](int r) { return r ^ (r >> 1 & 1); };

    // ---------------- two tiles at a time: their chains of products are independent
#pragma unroll 1
    while (used != fill) {
        const bool two = fill - used >= 2;
        const int4 e = *reinterpret_cast<const int4*>(&list[used % kList]);
        const uint8_t* tile[2] = {ring + ust * (2 * C::kChunk), ring + ust * (2 * C::kChunk) + (two ? C::kChunk : 0)};
        const int pos[2] = {e.y & ~15, (two ? e.w : e.y) & ~15};
        const bool partial = !two || ((e.y | e.w) & 1);
        copy_wait<C::kStages - 1>();
        __syncwarp();

        // ---------------- S^T = K Q^T
        float s[2][NT][4];
        {
            constexpr int W = D / 32;  // words of codes: D/8 bytes of the keys in places g and g + 8
            uint32_t kw[2][2][W], ku[2][2][D / 64];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int tok = order(g) + 8 * c;
                    const uint8_t* src = tile[u] + tok * (D / 2) + t * (D / 8);
                    const uint8_t* us = tile[u] + 8 * D + tok * (D / 16) + t * (D / 64);
                    if constexpr (D == 64) {
                        const uint2 v = *reinterpret_cast<const uint2*>(src);
                        kw[u][c][0] = v.x; kw[u][c][1] = v.y;
                    } else {
#pragma unroll
                        for (int i = 0; i < D / 128; ++i) {
                            const uint4 v = reinterpret_cast<const uint4*>(src)[i];
                            kw[u][c][4 * i] = v.x; kw[u][c][4 * i + 1] = v.y; kw[u][c][4 * i + 2] = v.z; kw[u][c][4 * i + 3] = v.w;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) ku[u][c][i] = us[i];
                }
#pragma unroll
            for (int w = 0; w < W; ++w) {  // a word: 8 dims, two steps
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t sc0 = scale2(ku[u][0][w / 2]), sc1 = scale2(ku[u][1][w / 2]);
                    uint32_t a[4], c[4];
                    decode_word(kw[u][0][w], a);
                    decode_word(kw[u][1][w], c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i] = mul2(a[i], sc0);
                        c[i] = mul2(c[i], sc1);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint2 q0 = sm.qf[n][2 * w][lane], q1 = sm.qf[n][2 * w + 1][lane];
                        if (w == 0) mma_first(s[u][n], a[0], c[0], a[1], c[1], q0.x, q0.y);
                        else mma(s[u][n], a[0], c[0], a[1], c[1], q0.x, q0.y);
                        mma(s[u][n], a[2], c[2], a[3], c[3], q1.x, q1.y);
                    }
                }
            }
        }

        // ---------------- V's bytes, to be there when the weights are
        constexpr int WV = D / 64;                // words of codes of a token: D/8 dims
        constexpr int B = D > 128 ? D / 128 : 1;  // blocks of those dims (D = 64: half of one)
        uint32_t vw[2][4][WV], vs[2][4][B];       // of the tokens in places 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int tok = order(2 * t + (c & 1)) + 8 * (c >> 1);
                const uint8_t* src = tile[u] + 9 * D + tok * (D / 2) + g * (D / 16);
                const uint8_t* us = tile[u] + 17 * D + tok * (D / 16);
                if constexpr (D == 64) {
                    vw[u][c][0] = *reinterpret_cast<const uint32_t*>(src);
                    vs[u][c][0] = us[g >> 1];
                } else if constexpr (D == 128) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    vw[u][c][0] = v.x; vw[u][c][1] = v.y;
                    vs[u][c][0] = us[g];
                } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(src);
                    vw[u][c][0] = v.x; vw[u][c][1] = v.y; vw[u][c][2] = v.z; vw[u][c][3] = v.w;
                    vs[u][c][0] = us[2 * g];
                    vs[u][c][B - 1] = us[2 * g + 1];
                }
            }

        // ---------------- scores less the rows' reference maxima, in log2 units; masked.
        // z[u][n][k]: rows (8 n + 2 t, + 1), place g + 8 k
        float2 z[2][NT][2], x[2][NT][2];
        if (MOD) {
            bool far = false;
            if (A.cap > 0.f) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float top[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        top[c] = max3(fmaxf(fabsf(s[0][n][c]), fabsf(s[0][n][c + 2])), fabsf(s[1][n][c]), fabsf(s[1][n][c + 2]));
                    far |= !(fabsf(top[0] * qs[n].x) < kNear * cap2 && fabsf(top[1] * qs[n].y) < kNear * cap2);
                }
                far = __any_sync(0xffffffffu, far);
            }
            auto each = [&](auto f) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) f(u, n, k);
            };
            each([&](int u, int n, int k) {
                x[u][n][k] = mul2f(make_float2(s[u][n][2 * k], s[u][n][2 * k + 1]), qs[n]);
                if (A.cap > 0.f) x[u][n][k] = capped(x[u][n][k], cap2, to_y, far);
            });
            // the biases; their origin moves first, and the maxima with it
            auto bias = [&](const float (&slope)[C::kRows], int moved, int origin) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float2 sl = *reinterpret_cast<const float2*>(&slope[8 * n + 2 * t]);
                    m[n] = fma2(sl, make_float2(-(float)moved, -(float)moved), m[n]);
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float at = (float)(pos[u] + order(g) + 8 * k - origin);
                            x[u][n][k] = fma2(sl, make_float2(at, at), x[u][n][k]);
                        }
                }
            };
            if (biased) {
                const int moved = max(max(pos[0], pos[1]) + (kTile - 1) - ref.x, 0);
                bias(sm.slope[0], moved, ref.x += moved);
            }
            if (below) {
                const int moved = min(min(pos[0], pos[1]) - ref.y, 0);
                bias(sm.slope[1], moved, ref.y += moved);
            }
            each([&](int u, int n, int k) { z[u][n][k] = make_float2(x[u][n][k].x - m[n].x, x[u][n][k].y - m[n].y); });
        } else {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        z[u][n][k] = fma2(make_float2(s[u][n][2 * k], s[u][n][2 * k + 1]), qs[n], make_float2(-m[n].x, -m[n].y));
        }
        auto mask = [&]() {  // -inf where a row does not see a key
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int p = pos[u] + order(g) + 8 * k;
                    const bool in = (u == 0 || two) && (!A.start || p >= start || p < prefix);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int2 at = *reinterpret_cast<const int2*>(&sm.qpos[8 * n + 2 * t]);
                        if (!in || p > at.x) z[u][n][k].x = -INFINITY;
                        if (!in || p > at.y) z[u][n][k].y = -INFINITY;
                    }
                }
        };
        if (partial) mask();
        bool more = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            // a NaN too moves the references: a key that is one, or -inf before the row's first key
            const float a = max3(z[0][n][0].x, z[0][n][0].y, z[0][n][1].x), b = max3(z[0][n][1].y, z[1][n][0].x, z[1][n][0].y);
            more |= !(max3(a, z[1][n][1].x, z[1][n][1].y) <= kRescale && b <= kRescale);
        }
        if (__any_sync(0xffffffffu, more)) {  // a row's maximum has grown: move every row's reference
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (!MOD) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int k = 0; k < 2; ++k) x[u][n][k] = mul2f(make_float2(s[u][n][2 * k], s[u][n][2 * k + 1]), qs[n]);
                }
                float2 top = m[n];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // a NaN counts as +inf, so that the joins keep the row; a masked key not at all
                        const float2 y = x[u][n][k], w = z[u][n][k];
                        if (w.x != -INFINITY) top.x = fmaxf(top.x, y.x == y.x ? y.x : INFINITY);
                        if (w.y != -INFINITY) top.y = fmaxf(top.y, y.y == y.y ? y.y : INFINITY);
                    }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, o));
                    top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, o));
                }
                const float2 f = make_float2(top.x > -INFINITY ? ex2(m[n].x - top.x) : 1.f, top.y > -INFINITY ? ex2(m[n].y - top.y) : 1.f);
                m[n] = top;
                l[n].x *= f.x;
                l[n].y *= f.y;
#pragma unroll
                for (int i = 0; i < C::kSteps; ++i) {
                    acc[i][n][0] *= f.x;
                    acc[i][n][1] *= f.y;
                    acc[i][n][2] *= f.x;
                    acc[i][n][3] *= f.y;
                }
                // a row without a key yet has m = -inf: its weights become 0, not NaN
                const float2 less = make_float2(top.x > -INFINITY ? top.x : 0.f, top.y > -INFINITY ? top.y : 0.f);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) z[u][n][k] = make_float2(x[u][n][k].x - less.x, x[u][n][k].y - less.y);
            }
            if (partial) mask();
        }
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 w = make_float2(ex2(z[u][n][k].x), ex2(z[u][n][k].y));
                    l[n] = add2(l[n], w);
                    pf[u][n][k] = transpose8x8(pack_half(w.x, w.y));
                }

        // ---------------- O^T += V^T P
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // a second tile that is not there has weights of zero
            if (partial) {
                // a key that no row sees may hold anything: its values become zeros, since a
                // weight of 0 would not undo a NaN. One that only later rows see has been
                // written, but its NaNs must not reach the rows before it: they are taken
                // out of the product and set in the outputs of the rows that see them.
                uint32_t nans = 0;  // bit 16 block + token
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int tok = order(2 * t + (c & 1)) + 8 * (c >> 1), p = pos[u] + tok;
                    const bool hidden = p >= length || (A.start && p < start && p >= prefix);
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        if (!hidden && vs[u][c][i] >= 0xF8u) nans |= (0x10000u * i + 1u - (uint32_t)i) << tok;
                        if (hidden || vs[u][c][i] >= 0xF8u) vs[u][c][i] = 0;
                    }
                }
                if (__any_sync(0xffffffffu, nans != 0)) {
                    nans |= __shfl_xor_sync(0xffffffffu, nans, 1);
                    nans |= __shfl_xor_sync(0xffffffffu, nans, 2);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int seen = sm.qpos[8 * n + 2 * t + c] - pos[u];  // the row sees tokens 0 .. seen of the tile
                            const uint32_t see = seen < 0 ? 0u : seen >= 15 ? 0xFFFFu : (2u << seen) - 1u;
#pragma unroll
                            for (int i = 0; i < C::kSteps; ++i)
                                if ((D == 256 && i >= C::kSteps / 2 ? nans >> 16 : nans) & see) acc[i][n][c] = acc[i][n][c + 2] = NAN;
                        }
                }
            }
#pragma unroll
            for (int w = 0; w < WV; ++w) {
                // two tokens' codes for one dimension into a byte, which decodes to the pair of
                // halves that the product takes: e their even dimensions, o the odd ones
                constexpr uint32_t kLow = 0x0F0F0F0Fu;
                uint32_t e[2][4], o[2][4];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t x = vw[u][2 * c][w], y = vw[u][2 * c + 1][w];
                    const uint32_t sc = vs[u][2 * c][w / 2] * 0x80u + (vs[u][2 * c + 1][w / 2] << 23);
                    decode_word((x & kLow) | (y << 4 & ~kLow), e[c]);
                    decode_word((x >> 4 & kLow) | (y & ~kLow), o[c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e[c][i] = mul2(e[c][i], sc);
                        o[c][i] = mul2(o[c][i], sc);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma(acc[4 * w + i][n], e[0][i], o[0][i], e[1][i], o[1][i], pf[u][n][0], pf[u][n][1]);
                }
            }
        }
        __syncwarp();  // every lane has read the stages: refill them
        used += two ? 2 : 1;
        ust = ust + 1 == C::kStages ? 0 : ust + 1;
        top_up();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---------------- join the warps: their outputs in the lanes' order, over the rings
    int2 last = ref;  // common origins
    auto reach = [&](const int2* of, int count) {  // of all of them, at most 32
        const int2 v = lane < count ? of[lane] : make_int2(0, INT_MAX);
        return make_int2(__reduce_max_sync(0xffffffffu, v.x), __reduce_min_sync(0xffffffffu, v.y));
    };
    auto shift = [&](float m, int r, int2 from) {
        return m - sm.slope[0][r] * (float)(last.x - from.x) - sm.slope[1][r] * (float)(last.y - from.y);
    };
    if (biased) {  // the maxima as from the common origins
        if (lane == 0) sm.wref[warp] = ref;
        __syncthreads();
        last = reach(sm.wref, warps);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + 2 * t;
            m[n] = make_float2(shift(m[n].x, r, ref), shift(m[n].y, r + 1, ref));
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, o);
            l[n].y += __shfl_xor_sync(0xffffffffu, l[n].y, o);
        }
        if (g == 0) *reinterpret_cast<float4*>(&sm.ml[warp][8 * n + 2 * t]) = make_float4(m[n].x, l[n].x, m[n].y, l[n].y);
    }
    constexpr int kFrags = C::kSteps * NT * 32, kItems = kFrags / 2;
    auto part = [&](int w) { return reinterpret_cast<float4*>(space + w * C::kSpace); };  // of a warp: [step][n][lane]
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            part(warp)[(i * NT + n) * 32 + lane] = make_float4(acc[i][n][0], acc[i][n][1], acc[i][n][2], acc[i][n][3]);
    __syncthreads();

    // The sum of partial results of item x -- steps 2 j, 2 j + 1 of a lane: 4 dimensions of rows
    // r, r + 1 -- relative to their largest maxima, kBatch of them at a time (their loads are
    // all on their way before the first is used).
    struct Joined {
        float4 a, b;      // steps 2 j and 2 j + 1
        float2 top, sum;  // of rows r and r + 1
    };
    constexpr int kBatch = 4;
    auto join = [&](int x, int count, auto ml_of, auto frag_of) {
        const int n = x / 32 % NT, r = 8 * n + 2 * (x & 3);
        Joined o;
        o.a = o.b = make_float4(0.f, 0.f, 0.f, 0.f);
        o.top = make_float2(-INFINITY, -INFINITY);
        o.sum = make_float2(0.f, 0.f);
        for (int w0 = 0; w0 < count; w0 += kBatch) {
            float4 v[kBatch], a[kBatch], c[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int w = min(w0 + i, count - 1);
                v[i] = ml_of(w, r);
                a[i] = frag_of(w, x, 0);
                c[i] = frag_of(w, x, 1);
            }
            float2 top = o.top;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (w0 + i >= count) v[i].x = v[i].z = -INFINITY;
                top = make_float2(fmaxf(top.x, v[i].x), fmaxf(top.y, v[i].z));
            }
            // -inf: no key of the row there
            const float ox = o.top.x == -INFINITY ? 0.f : ex2(o.top.x - top.x), oy = o.top.y == -INFINITY ? 0.f : ex2(o.top.y - top.y);
            o.top = top;
            o.sum = make_float2(o.sum.x * ox, o.sum.y * oy);
            o.a = make_float4(o.a.x * ox, o.a.y * oy, o.a.z * ox, o.a.w * oy);
            o.b = make_float4(o.b.x * ox, o.b.y * oy, o.b.z * ox, o.b.w * oy);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float fx = v[i].x == -INFINITY ? 0.f : ex2(v[i].x - top.x), fy = v[i].z == -INFINITY ? 0.f : ex2(v[i].z - top.y);
                o.sum.x += fx * v[i].y;
                o.sum.y += fy * v[i].w;
                o.a.x += fx * a[i].x; o.a.y += fy * a[i].y; o.a.z += fx * a[i].z; o.a.w += fy * a[i].w;
                o.b.x += fx * c[i].x; o.b.y += fy * c[i].y; o.b.z += fx * c[i].z; o.b.w += fy * c[i].w;
            }
        }
        return o;
    };
    auto write = [&](int x, const Joined& o) {
        const int ln = x & 31, n = x / 32 % NT, j = x / 32 / NT, r = 8 * n + 2 * (ln & 3), d = (ln >> 2) * (D / 8) + 4 * j;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int row = r0 + r + c;
            if (row >= rows) break;
            const int tok = P.group(row), head = h * A.G + row - tok * A.G;
            const float top = c ? o.top.y : o.top.x, sum = c ? o.sum.y : o.sum.x, inv = top > -INFINITY ? rcp(sum) : 0.f;
            const float y0 = (c ? o.a.y : o.a.x) * inv, y1 = (c ? o.a.w : o.a.z) * inv, y2 = (c ? o.b.y : o.b.x) * inv,
                        y3 = (c ? o.b.w : o.b.z) * inv;
            uint2 w;
            if (bf16) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(y0, y1), hi = __floats2bfloat162_rn(y2, y3);
                w = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            } else {
                w = make_uint2(pack_half(y0, y1), pack_half(y2, y3));
            }
            *reinterpret_cast<uint2*>(A.o + b * A.o_batch + tok * A.o_token + head * A.o_head + d) = w;
            if (d == 0) {
                float e = -INFINITY;
                if (top > -INFINITY) {
                    e = (top + lg2(sum)) * kLn2;
                    if (biased) {
                        const float sl = load(A.slopes + head);
                        e -= sl * (float)(qpos0 + tok - (sl < 0.f ? last.y : last.x));
                    }
                }
                A.lse[((size_t)b * A.Tq + tok) * A.H * A.G + head] = e;
            }
        }
    };
    auto warp_ml = [&](int w, int r) { return *reinterpret_cast<const float4*>(&sm.ml[w][r]); };
    auto warp_frag = [&](int w, int x, int k) { return part(w)[((2 * (x / 32 / NT) + k) * NT + x / 32 % NT) * 32 + (x & 31)]; };
    if (nsplit == 1) {
        for (int x = tid; x < kItems; x += threads) write(x, join(x, warps, warp_ml, warp_frag));
        return;
    }
    // ---------------- join the shares: item x is sent to CTA x % nsplit, which joins and writes it
    const int per = (kItems + nsplit - 1) / nsplit;
    float4* frags = reinterpret_cast<float4*>(space + warps * C::kSpace);  // [share][item / nsplit][2]
    cluster_wait();
    for (int x = tid; x < kItems; x += threads) {
        const Joined o = join(x, warps, warp_ml, warp_frag);
        const int ix = P.shares(x), to = x - ix * nsplit;
        peer_store(frags + (split * per + ix) * 2, to, o.a);
        peer_store(frags + (split * per + ix) * 2 + 1, to, o.b);
        if (x / 32 / NT == 0 && (x & 31) < 4)  // the row pair's first item
            for (int s = 0; s < nsplit; ++s)
                peer_store(reinterpret_cast<float4*>(&sm.xml[split][8 * (x / 32) + 2 * (x & 3)]), s, make_float4(o.top.x, o.sum.x, o.top.y, o.sum.y));
    }
    if (biased && tid < nsplit) peer_store(&sm.xref[split], tid, last);
    cluster_arrive();
    cluster_wait();
    if (biased) {
        last = reach(sm.xref, nsplit);
        for (int i = tid; i < nsplit * C::kRows; i += threads) {
            const int share = i / C::kRows, r = i % C::kRows;
            sm.xml[share][r].x = shift(sm.xml[share][r].x, r, sm.xref[share]);
        }
        __syncthreads();
    }
    for (int ix = tid; ix * nsplit + split < kItems; ix += threads)
        write(ix * nsplit + split, join(ix * nsplit + split, nsplit, [&](int s, int r) { return *reinterpret_cast<const float4*>(&sm.xml[s][r]); },
                                        [&](int s, int, int k) { return frags[(s * per + ix) * 2 + k]; }));
}

// How many clusters of n CTAs of 4 w warps the device holds at once, by [w - 1][n - 1].
struct Room {
    int clusters[kMaxWarps / 4][kMaxSplit];
};

template <int D, int NT, bool MOD>
cudaError_t set_up(Room* room) {
    const auto kernel = attend_pages_kernel<D, NT, MOD>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Config<D, NT>::smem(Config<D, NT>::kSmWarps, kMaxSplit));
    for (int w = 1; e == cudaSuccess && 4 * w <= Config<D, NT>::kSmWarps; ++w)
        for (int n = 1; e == cudaSuccess && n <= kMaxSplit; ++n) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(n);
            cfg.blockDim = dim3(4 * w * 32);
            cfg.dynamicSmemBytes = Config<D, NT>::smem(4 * w, n);
            cudaLaunchAttribute at;
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = n;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            cfg.attrs = &at;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&room->clusters[w - 1][n - 1], kernel, &cfg);
        }
    return e;
}

// Warps of a CTA, CTAs that share a selection and jobs that are not shared: what has the least
// estimated time, in cycles, the larger of two bounds. Work: a tile takes an SM about `tile`
// (what its instructions cost at the rate reached with many warps), a warp's start and end 450,
// a shared CTA's join 1600 more. Chain: a warp's own pairs of tiles follow each other at `pair`
// behind 4500 of start and end (1000 more if shared), and again for the CTAs that find no room
// at first. With few jobs the chain decides and more, smaller shares win; with many the work
// does, and shares only cost, but for the jobs that some SMs have more of than others. us a call:
//   1 request, 8 heads, 128 tiles:    8 CTAs of 8 warps 5.2, of 4 warps 5.5, of 12 warps 6.4
//   16 jobs of 512 tiles, 16 rows:    6 CTAs of 12 warps 15.2, of 8 warps 15.7, 7 of 12 27.0
//   256 jobs of 128 tiles, 32 rows:   whole 38.2, 152 whole and 104 halved 46.7, all halved 46.8
//   512 jobs of 128 tiles:            whole 34.5, all halved 35.6, 456 whole and 56 halved 32.9;
//                                     such mixtures in clusters of 3, 4 or 8: 37.0, 34.1, 35.2
// The constants are fitted to the times of every split of 110 calls (heads of 64, 128 and 256,
// 1 to 64 rows, 8 to 2000 jobs of 8 to 1200 tiles): the split taken is 1.2 % slower than the best one
// on average and 16 % at most.
void plan(const Room& room, int sm_warps, int num_sms, int D, int NT, int64_t jobs, int64_t tiles, int* warps, int* shares,
          int64_t* whole) {
    const float tile = 7.f + 0.55f * D + NT * (10.f + 0.12f * D), pair = 2000.f + 290.f / 128 * NT * D;
    float best = INFINITY;
    *warps = 4;
    *shares = 1;
    *whole = jobs;
    for (int n = 1; n <= kMaxSplit; ++n)
        for (int w = 4; w <= sm_warps; w += 4) {
            const int64_t fit = (int64_t)room.clusters[w / 4 - 1][n - 1] * n;  // CTAs
            if (fit < 1 || ((n > 1 || w > 4) && 2 * (int64_t)n * w > tiles)) continue;
            const float share = (float)tiles / n, ends = n > 1 ? 5500.f : 4500.f;
            const float work_1 = tiles * tile + 450.f * w, work_n = share * tile + 450.f * w + (n > 1 ? 1600.f : 0.f);
            const float chain_1 = ends + ceilf((float)tiles / (2 * w)) * pair, chain_n = ends + ceilf(share / (2 * w)) * pair;
            auto consider = [&](float work, float chain, int64_t alone) {
                if (fmaxf(work, chain) >= best) return;
                best = fmaxf(work, chain);
                *warps = w;
                *shares = n;
                *whole = alone;
            };
            const float ctas = (float)jobs * n;
            consider(ceilf(ctas / num_sms) * work_n, ceilf(ctas / fit) * chain_n, n == 1 ? jobs : 0);
            // as many whole jobs as every SM can have alike, the others halved
            const int64_t even = n == 2 ? jobs / num_sms * num_sms / n * n : 0;
            if (even == 0) continue;
            const float halves = (float)(jobs - even) * n;
            consider((float)(even / num_sms) * work_1 + ceilf(halves / num_sms) * work_n,
                     chain_1 + (even + halves > fit ? chain_n : 0.f), even);
        }
}

template <int D, int NT, bool MOD>
cudaError_t launch(cudaStream_t stream, bool bf16, const PageAttention& a, int num_sms) {
    using C = Config<D, NT>;
    static PerDevice<Room> rooms;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= PerDevice<Room>::kDevices) return cudaErrorInvalidDevice;
    const Room* room = nullptr;
    if ((e = (cudaError_t)rooms.get(dev, set_up<D, NT, MOD>, &room)) != cudaSuccess) return e;
    const int row_tiles = (a.G * a.Tq + C::kRows - 1) / C::kRows;
    const int64_t jobs = (int64_t)a.B * a.H * row_tiles, tiles = (int64_t)a.k * a.tiles;
    int warps, shares;
    int64_t whole;  // jobs that are not shared, a multiple of shares
    plan(*room, C::kSmWarps, num_sms, D, NT, jobs, tiles, &warps, &shares, &whole);
    const int64_t ctas = whole + (jobs - whole) * shares;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    Split p;
    p.shares = Divisor(shares);
    p.row_tiles = Divisor(row_tiles);
    p.heads = Divisor(a.H);
    p.tiles = Divisor(a.tiles);
    p.group = Divisor(a.G);
    p.whole = (int)(whole / shares);
    p.ntiles = (int)tiles;
    p.groups = (int)((tiles + 32 * shares * warps - 1) / (32 * shares * warps));
    p.groups_1 = (int)((tiles + 32 * warps - 1) / (32 * warps));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = C::smem(warps, shares);
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)shares;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, attend_pages_kernel<D, NT, MOD>, a, p, bf16);
}

template <int D, bool MOD>
cudaError_t by_rows(cudaStream_t stream, bool bf16, const PageAttention& a, int num_sms) {
    const int rows = a.G * a.Tq;
    if (rows <= 8) return launch<D, 1, MOD>(stream, bf16, a, num_sms);
    if constexpr (D < 256)  // at 256 the outputs of 32 rows would fill the register file
        if (rows > 16) return launch<D, 4, MOD>(stream, bf16, a, num_sms);
    return launch<D, 2, MOD>(stream, bf16, a, num_sms);
}

template <int D>
cudaError_t by_scores(cudaStream_t stream, bool bf16, const PageAttention& a, int num_sms) {
    return a.cap > 0.f || a.slopes ? by_rows<D, true>(stream, bf16, a, num_sms) : by_rows<D, false>(stream, bf16, a, num_sms);
}

}  // namespace

cudaError_t launch_attend_pages(cudaStream_t stream, const PageShape& ps, bool bf16, const PageAttention& a, int num_sms) {
    if (a.B == 0) return cudaSuccess;
    if (ps.dim == 64) return by_scores<64>(stream, bf16, a, num_sms);
    if (ps.dim == 128) return by_scores<128>(stream, bf16, a, num_sms);
    return by_scores<256>(stream, bf16, a, num_sms);
}

}  // namespace hs
