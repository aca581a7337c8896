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
// What bounds it: each key and head costs 9/8 D bytes of HBM and 4 D multiply-adds a row, so
// up to about 16 rows the stream of pages is the floor, and the work per byte -- two
// conversions, two scalings and half a register shuffle for each pair of codes -- has to stay
// under it. So nothing decoded goes through shared memory: a warp decodes its tile's codes
// straight into the registers in which the tensor cores (mma.sync m16n8k16, f16 operands, f32
// sums) take them. Both products are formed transposed, keys (or dimensions) along the 16
// rows of the instruction and the query rows along its 8 columns, so that a group of up to 8
// query rows costs one instruction where the other way round would pad it to 16.
//
// Work split: one CTA per (request, KV head, tile of query rows, share of the selection); a
// selection is shared by up to 8 CTAs, one thread-block cluster, when there are few requests
// and heads. Each of the CTA's warps takes 16-token tiles in turn (18 D contiguous bytes: one
// bulk copy into the warp's own ring of stages, no barrier between warps) and keeps its own
// maxima, sums and outputs; the warps are joined through shared memory at the end and the
// CTAs of a cluster through distributed shared memory, so no workspace and no second kernel.
//
//   S^T = K Q^T  A: 16 keys x 16 dims. Which 4 dimensions a lane holds at a step is free as
//                long as Q's do the same: lane (g, t) = (lane / 4, lane % 4) takes dimensions
//                t D/4 + 4 i ... of keys g and g + 8 at step i, so its codes are D/8
//                contiguous bytes of a row and its scales D/64 bytes.
//   O^T = V^T P  A: 16 dims x 16 keys. Lane (g, t) needs pairs of keys (2t, 2t+1) and (2t+8,
//                2t+9) for the same dimension: it decodes the same bytes of four tokens and
//                interleaves them. At step i it holds dimensions g D/8 + 2 i and + 1.
//   P            leaves S^T's layout (a lane has keys g, g + 8 of rows 2t, 2t + 1) for the
//                other operand's (keys 2t, 2t + 1 of row g) by a transposing register move.
//
// Decoded keys and values are exact halves (hs_page.cu). Queries become halves too: fp16 ones
// as they are, bf16 ones scaled per row by a power of two that brings the row's largest
// magnitude to [2^13, 2^14), which keeps all eight bits of every component down to 2^-27 of
// the largest; what is below is rounded by at most 2^-38 of the largest. Softmax weights are
// rounded to half (2^-11 relative, unless below 2^-14 of the largest) for the second product
// only; the sums that normalise them add the unrounded ones in f32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "hs_page.h"

namespace hs {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kMaxSplit = 8;           // CTAs that share a selection: the portable cluster size
constexpr int kList = 64;              // a warp's list of live tiles (a ring; 32 are added at a time)
constexpr float kRescale = 8.f;        // a row's reference maximum moves when exceeded by 2^8
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

template <int D, int NT>
struct Config {
    static constexpr int kChunk = 18 * D;           // bytes of a tile of one head
    static constexpr int kRows = 8 * NT;            // query rows of a CTA
    static constexpr int kSteps = D / 16;
    static constexpr int kCtas = NT * D <= 128 ? 4 : NT * D <= 256 ? 3 : 2;  // CTAs an SM: registers
    static constexpr int kStages = D == 64 ? 6 : D == 128 ? 4 : 3;
    static constexpr int kRing = kWarps * kStages * kChunk;
    static constexpr int kPart = kWarps * kRows * D * 4;  // the warps' outputs, over the ring
    static constexpr int kSpace = kRing > kPart ? kRing : kPart;
};

template <int D, int NT>
struct Smem {
    using C = Config<D, NT>;
    alignas(128) uint8_t space[C::kSpace];
    uint2 qf[NT][C::kSteps][32];              // Q as the lanes take it
    alignas(16) float joined[C::kRows][D];    // this CTA's output, relative to its maxima
    float qscale[C::kRows], slope[C::kRows];  // of the rows: to log2 units
    int qpos[C::kRows];
    float m[kWarps][C::kRows], l[kWarps][C::kRows];
    float f[kMaxSplit][C::kRows];             // factors of the warps, then of the shares
    float cm[C::kRows], cl[C::kRows];         // this CTA's maxima and sums
    float pm[kMaxSplit][C::kRows], pl[kMaxSplit][C::kRows];  // every share's
    float inv[C::kRows];
    int wref[kWarps], cref;                   // positions that biases are relative to
    uint64_t bar[kWarps][C::kStages];
    int2 list[kWarps][kList];                 // unit (slot * tiles + tile), position | partial
};

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
// tanh y = 1 - 2 / (1 + e^(2y)); y2 = 2 y log2 e. Absolute error a few 2^-23.
__device__ __forceinline__ float tanh_of(float y2) { return 1.f - __fdividef(2.f, 1.f + ex2(y2 > 100.f ? 100.f : y2)); }

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
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(su32(b)), "r"(parity) : "memory");
    return ok != 0;
}
// Waits for a copy to land; gives up once the global timer passes `deadline`.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, uint64_t deadline) {
    while (!bar_try(b, parity))
        if (global_ns() > deadline) return false;
    return true;
}
// `bytes` (a multiple of 16, both ends 16-byte aligned) into shared memory, counted on `b`.
__device__ __forceinline__ void copy_in(void* dst, const uint8_t* src, uint32_t bytes, uint64_t* b) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(su32(dst)),
                 "l"(src), "r"(bytes), "r"(su32(b))
                 : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned; barrier.cluster.wait.aligned;" ::: "memory");
}
// A float of another CTA of the cluster, at the place of this CTA's `p`.
__device__ __forceinline__ float peer_float(const float* p, int rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(su32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 peer_float4(const float* p, int rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(su32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ int peer_int(const int* p, int rank) {
    return __float_as_int(peer_float(reinterpret_cast<const float*>(p), rank));
}

// MOD: scores are capped or biased.
template <int D, int NT, bool MOD>
__global__ void __launch_bounds__(kThreads, (Config<D, NT>::kCtas)) attend_pages_kernel(const PageAttention A, int nsplit, int row_tiles, bool bf16) {
    using C = Config<D, NT>;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem<D, NT>& sm = *reinterpret_cast<Smem<D, NT>*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint64_t deadline = global_ns() + A.wait_ns;
    int job = blockIdx.x / nsplit;
    const int split = blockIdx.x - job * nsplit;  // = the rank in the cluster
    const int rt = job % row_tiles;
    job /= row_tiles;
    const int b = job / A.H, h = job - b * A.H;
    const int rows = A.G * A.Tq, r0 = rt * C::kRows;

    // ---------------- this warp's tiles: every (nsplit * kWarps)-th of the selection. Lane i
    // looks up the i-th of the next 32; those that hold a visible key go on the warp's list.
    const int32_t* slots = A.slots + (size_t)b * A.k;
    const int32_t* sel = A.sel + (size_t)b * A.k;
    const int ntiles = A.k * A.tiles, stride = nsplit * kWarps;
    int next = lane * stride + split * kWarps + warp;  // this lane's tile of the next group
    int gslot = -1, gsel = -1;                          // its page, loaded a group ahead
    auto look_up = [&]() {
        gslot = -1;
        if (next < ntiles) {
            const int j = next / A.tiles;
            gslot = __ldg(slots + j);
            gsel = __ldg(sel + j);
        }
    };
    look_up();
    // the request's mask: query token t sees p <= length - Tq + t and (p >= start or p < prefix)
    const int length = __ldg(A.lengths + b);
    const int start = A.start ? __ldg(A.start + b) : 0;
    const int prefix = A.prefix ? __ldg(A.prefix + b) : 0;
    const int qpos0 = length - A.Tq;  // may be negative
    const uint8_t* pages = A.pages + ((size_t)b * A.S * A.tiles * A.H + h) * C::kChunk;
    const size_t unit_bytes = (size_t)A.H * C::kChunk;

    uint8_t* ring = sm.space + warp * (C::kStages * C::kChunk);
    uint64_t* bar = sm.bar[warp];
    int2* list = sm.list[warp];
    if (lane < C::kStages) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(su32(bar + lane)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();

    int groups = (ntiles + 32 * stride - 1) / (32 * stride);  // not yet on the list
    uint32_t used = 0, fill = 0, tail = 0;  // listed tiles consumed, copied (or on their way), listed
    auto append = [&]() {
        bool live = false;
        int2 e;
        if (gslot >= A.S && A.status) atomicOr(A.status, 1u /* HS_STATUS_RANGE */);
        if (gslot >= 0 && gslot < A.S && gsel >= 0) {
            const int tile = next % A.tiles;
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
    auto top_up = [&]() {  // keep every stage on its way
        while (fill - used < C::kStages) {
            if (fill == tail) {
                if (groups == 0) break;
                append();
                continue;
            }
            if (lane == 0) {
                const int st = fill % C::kStages;
                copy_in(ring + st * C::kChunk, pages + (size_t)list[fill % kList].x * unit_bytes, C::kChunk, &bar[st]);
            }
            ++fill;
        }
    };
    top_up();

    // ---------------- the query rows as halves, in the lanes' order
    for (int r = warp; r < C::kRows; r += kWarps) {
        constexpr int N = D / 32;
        const int row = r0 + r;
        float x[N], scale = 0.f;
        if (row < rows) {
            const int tok = row / A.G, head = h * A.G + row - tok * A.G;
            const uint16_t* src = A.q + b * A.q_batch + tok * A.q_token + head * A.q_head + lane * N;
            uint32_t w[N / 2];
            if constexpr (N == 2) {
                w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
            } else if constexpr (N == 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
                w[0] = v.x; w[1] = v.y;
            } else {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            }
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t u = w[i / 2] >> (16 * (i & 1)) & 0xFFFFu;
                x[i] = bf16 ? __uint_as_float(u << 16) : __half2float(__ushort_as_half((uint16_t)u));
                amax = fmaxf(amax, fabsf(x[i]));
            }
            scale = 1.f;
            if (bf16) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                if (amax > 0.f && amax < INFINITY) {
                    const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 13, -100);
                    scale = __uint_as_float((uint32_t)(127 + e) << 23);
                    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                    for (int i = 0; i < N; ++i) x[i] *= inv;
                }
            }
            if (lane == 0) {
                // to log2 units; with a cap, to 2 log2 e s / cap
                sm.qscale[r] = MOD && A.cap > 0.f ? scale * (A.scale * (2.f * kLog2e / A.cap)) : scale * (A.scale * kLog2e);
                sm.slope[r] = MOD && A.slopes ? __ldg(A.slopes + head) * kLog2e : 0.f;
                sm.qpos[r] = qpos0 + tok;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = 0.f;
            if (lane == 0) {
                sm.qscale[r] = sm.slope[r] = 0.f;
                sm.qpos[r] = qpos0;
            }
        }
        // dimension d is taken by lane t = d / (D/4) of row r's group at step d % (D/4) / 4
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const int d = lane * N + i, dt = d / (D / 4), step = d % (D / 4) / 4;
            reinterpret_cast<uint32_t*>(&sm.qf[r / 8][step][(r % 8) * 4 + dt])[d % 4 / 2] = pack_half(x[i], x[i + 1]);
        }
    }
    __syncthreads();

    constexpr bool kKeepQ = NT == 1 && D <= 128;  // Q in registers
    uint2 qreg[kKeepQ ? C::kSteps : 1];
    if (kKeepQ) {
#pragma unroll
        for (int i = 0; i < C::kSteps; ++i) qreg[kKeepQ ? i : 0] = sm.qf[0][i][lane];
    }
    float2 qs[NT];  // rows 8 n + 2 t, + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) qs[n] = *reinterpret_cast<const float2*>(&sm.qscale[8 * n + 2 * t]);
    const float cap2 = A.cap * kLog2e;

    float acc[C::kSteps][NT][4];  // O^T: dims g D/8 + 2 i (c = 0, 1), + 1 (2, 3); rows 8 n + 2 t, + 1
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < C::kSteps; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][n][c] = 0.f;
    }
    int ref = 0;  // biases are relative to this position: the last of the tiles so far
    // The order of a tile's keys along the instruction: place r holds token order(r). A lane's
    // four tokens of V (places 2t, 2t + 1, + 8) then lie in both halves of the 128 bytes that
    // the shared memory banks cover, and its keys still do.
    auto order = [](int r) { return r ^ (r >> 1 & 1); };
    bool ok = true;

    // ---------------- two tiles at a time: their chains of products are independent
#pragma unroll 1
    while (used != fill) {
        const bool two = fill - used >= 2;
        const uint8_t* tile[2];
        int pos[2];
        bool partial = !two;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t at = used + (two ? u : 0), st = at % C::kStages;
            tile[u] = ring + st * C::kChunk;
            const int word = list[at % kList].y;
            pos[u] = word & ~15;
            partial |= word & 1;
            if (!__all_sync(0xffffffffu, bar_wait(&bar[st], (at / C::kStages) & 1u, deadline))) ok = false;
        }
        if (!ok) break;

        // ---------------- S^T = K Q^T
        float s[2][NT][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.f;
        {
            constexpr int W = D / 32;  // words of codes: D/8 bytes of the keys in places g and g + 8
            uint32_t kw[2][2][W], ku[2][2];
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
                        ku[u][c] = *us;
                    } else {
#pragma unroll
                        for (int i = 0; i < D / 128; ++i) {
                            const uint4 v = reinterpret_cast<const uint4*>(src)[i];
                            kw[u][c][4 * i] = v.x; kw[u][c][4 * i + 1] = v.y; kw[u][c][4 * i + 2] = v.z; kw[u][c][4 * i + 3] = v.w;
                        }
                        ku[u][c] = D == 128 ? *reinterpret_cast<const uint16_t*>(us) : *reinterpret_cast<const uint32_t*>(us);
                    }
                }
#pragma unroll
            for (int w = 0; w < W; ++w) {  // a word: 8 dims, two steps
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t sc0 = scale2(ku[u][0] >> (8 * (w / 2)) & 0xFFu), sc1 = scale2(ku[u][1] >> (8 * (w / 2)) & 0xFFu);
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
                        const uint2 q0 = kKeepQ ? qreg[kKeepQ ? 2 * w : 0] : sm.qf[n][2 * w][lane];
                        const uint2 q1 = kKeepQ ? qreg[kKeepQ ? 2 * w + 1 : 0] : sm.qf[n][2 * w + 1][lane];
                        mma(s[u][n], a[0], c[0], a[1], c[1], q0.x, q0.y);
                        mma(s[u][n], a[2], c[2], a[3], c[3], q1.x, q1.y);
                    }
                }
            }
        }

        // ---------------- scores in log2 units, masked; s[u][n][c + 2 k]: row c, place g + 8 k
        if (MOD) {
            const int last = max(pos[0], pos[1]) + (kTile - 1), moved = last - ref;
            if (A.slopes && moved > 0) {  // move the origin of the biases
                ref = last;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) m[n][c] -= sm.slope[8 * n + 2 * t + c] * (float)moved;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 sl = *reinterpret_cast<const float2*>(&sm.slope[8 * n + 2 * t]);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float y = s[u][n][c] * (c & 1 ? qs[n].y : qs[n].x);
                        if (A.cap > 0.f) y = cap2 * tanh_of(y);
                        s[u][n][c] = y - (c & 1 ? sl.y : sl.x) * (float)(ref - (pos[u] + order(g) + 8 * (c >> 1)));
                    }
            }
        } else {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[u][n][c] *= c & 1 ? qs[n].y : qs[n].x;
        }
        if (partial) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int p = pos[u] + order(g) + 8 * k;
                    const bool in = (u == 0 || two) && (!A.start || p >= start || p < prefix);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (!in || p > sm.qpos[8 * n + 2 * t + c]) s[u][n][c + 2 * k] = -INFINITY;
                }
        }
        bool more = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                more |= !(fmaxf(fmaxf(s[0][n][c], s[0][n][c + 2]), fmaxf(s[1][n][c], s[1][n][c + 2])) <= m[n][c] + kRescale);
        if (__any_sync(0xffffffffu, more)) {  // a row's maximum has grown: move every row's reference
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = m[n][c];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {  // a NaN counts as +inf, so that the joins keep the row
                            const float y = s[u][n][c + 2 * k];
                            top = fmaxf(top, y == y ? y : INFINITY);
                        }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const float f = top > -INFINITY ? ex2(m[n][c] - top) : 1.f;
                    m[n][c] = top;
                    l[n][c] *= f;
#pragma unroll
                    for (int i = 0; i < C::kSteps; ++i) {
                        acc[i][n][c] *= f;
                        acc[i][n][c + 2] *= f;
                    }
                }
        }
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    w[c] = ex2(s[u][n][c] - m[n][c & 1]);
                    if (partial && s[u][n][c] == -INFINITY) w[c] = 0.f;  // m is -inf too in a row without a key yet
                }
                l[n][0] += w[0] + w[2];
                l[n][1] += w[1] + w[3];
                pf[u][n][0] = transpose8x8(pack_half(w[0], w[1]));
                pf[u][n][1] = transpose8x8(pack_half(w[2], w[3]));
            }

        // ---------------- O^T += V^T P
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (u == 1 && !two) break;
            constexpr int W = D / 64;  // words of codes of a token: D/8 dims
            uint32_t vw[4][W], vs[4];  // of the tokens in places 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int tok = order(2 * t + (c & 1)) + 8 * (c >> 1);
                const uint8_t* src = tile[u] + 9 * D + tok * (D / 2) + g * (D / 16);
                const uint8_t* us = tile[u] + 17 * D + tok * (D / 16);
                if constexpr (D == 64) {
                    vw[c][0] = *reinterpret_cast<const uint32_t*>(src);
                    vs[c] = us[g >> 1];
                } else if constexpr (D == 128) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    vw[c][0] = v.x; vw[c][1] = v.y;
                    vs[c] = us[g];
                } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(src);
                    vw[c][0] = v.x; vw[c][1] = v.y; vw[c][2] = v.z; vw[c][3] = v.w;
                    vs[c] = *reinterpret_cast<const uint16_t*>(us + 2 * g);
                }
            }
            if (partial) {
                // a key that no row sees may hold anything: its values become zeros, since a
                // weight of 0 would not undo a NaN. One that only later rows see has been
                // written, but its NaNs must not reach the rows before it: they are taken
                // out of the product and set in the outputs of the rows that see them.
                uint32_t nans = 0;  // bit 16 (half of the dims) + token
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int tok = order(2 * t + (c & 1)) + 8 * (c >> 1), p = pos[u] + tok;
                    if (p >= length || (A.start && p < start && p >= prefix)) vs[c] = 0;
                    if ((vs[c] & 0xFFu) >= 0xF8u) { vs[c] &= 0xFF00u; nans |= 1u << tok; }
                    if (D == 256 && vs[c] >= 0xF800u) { vs[c] &= 0xFFu; nans |= 0x10000u << tok; }
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
            for (int w = 0; w < W; ++w) {
                uint32_t d[4][4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    decode_word(vw[c][w], d[c]);
                    const uint32_t sc = scale2(D == 256 ? vs[c] >> (8 * (w / 2)) & 0xFFu : vs[c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[c][i] = mul2(d[c][i], sc);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = prmt(d[0][i], d[1][i], 0x5410), a1 = prmt(d[0][i], d[1][i], 0x7632);
                    const uint32_t a2 = prmt(d[2][i], d[3][i], 0x5410), a3 = prmt(d[2][i], d[3][i], 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma(acc[4 * w + i][n], a0, a1, a2, a3, pf[u][n][0], pf[u][n][1]);
                }
            }
        }
        __syncwarp();  // every lane has read the stages: refill them
        used += two ? 2 : 1;
        top_up();
    }
    if (!ok) {
        if (A.status && lane == 0) atomicOr(A.status, 8u /* HS_STATUS_TIMEOUT */);
        // no copy may still be landing when the CTA exits: wait for them, bounded again
        const uint64_t by = global_ns() + kDefaultWaitNs;
        for (; used != fill; ++used) bar_wait(&bar[used % C::kStages], (used / C::kStages) & 1u, by);
    }

    // ---------------- join the warps: their outputs in the lanes' order, over the ring
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float sum = l[n][c];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (g == 0) {
                sm.m[warp][8 * n + 2 * t + c] = m[n][c];
                sm.l[warp][8 * n + 2 * t + c] = sum;
            }
        }
    if (lane == 0) sm.wref[warp] = ref;
    __syncthreads();  // every warp is done with its ring
    constexpr int kFrags = C::kSteps * NT * 32;
    float4* part = reinterpret_cast<float4*>(sm.space);  // [warp][step][n][lane]
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            part[warp * kFrags + (i * NT + n) * 32 + lane] = make_float4(acc[i][n][0], acc[i][n][1], acc[i][n][2], acc[i][n][3]);
    if (tid < C::kRows) {
        int last = sm.wref[0];
        if (MOD)
            for (int w = 1; w < kWarps; ++w) last = max(last, sm.wref[w]);
        float mw[kWarps], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mw[w] = sm.m[w][tid];
            if (MOD) mw[w] -= sm.slope[tid] * (float)(last - sm.wref[w]);
            top = fmaxf(top, mw[w]);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = mw[w] == -INFINITY ? 0.f : ex2(mw[w] - top);  // -inf: the warp saw no key of the row
            sm.f[w][tid] = f;
            sum += f * sm.l[w][tid];
        }
        sm.cm[tid] = top;
        sm.cl[tid] = sum;
        sm.inv[tid] = top > -INFINITY ? 1.f / sum : 0.f;
        if (tid == 0) sm.cref = last;
    }
    __syncthreads();
    for (int x = tid; x < kFrags; x += kThreads) {
        const int ln = x % 32, n = x / 32 % NT, i = x / 32 / NT, r = 8 * n + 2 * (ln & 3), d = (ln >> 2) * (D / 8) + 2 * i;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 v = part[w * kFrags + x];
            const float2 f = *reinterpret_cast<const float2*>(&sm.f[w][r]);
            o.x += f.x * v.x; o.y += f.y * v.y; o.z += f.x * v.z; o.w += f.y * v.w;
        }
        *reinterpret_cast<float2*>(&sm.joined[r][d]) = make_float2(o.x, o.z);
        *reinterpret_cast<float2*>(&sm.joined[r + 1][d]) = make_float2(o.y, o.w);
    }
    // ---------------- join the shares, each CTA a part of the rows' elements, and write
    int last = 0;
    if (nsplit > 1) {
        cluster_sync();
        if (MOD) {
            last = sm.cref;
            for (int s = 0; s < nsplit; ++s) last = max(last, peer_int(&sm.cref, s));
        }
        for (int x = tid; x < nsplit * C::kRows; x += kThreads) {
            const int s = x / C::kRows, r = x % C::kRows;
            float ms = peer_float(&sm.cm[r], s);
            if (MOD) ms -= sm.slope[r] * (float)(last - peer_int(&sm.cref, s));
            sm.pm[s][r] = ms;
            sm.pl[s][r] = peer_float(&sm.cl[r], s);
        }
        __syncthreads();
        if (tid < C::kRows) {
            float top = -INFINITY, sum = 0.f;
            for (int s = 0; s < nsplit; ++s) top = fmaxf(top, sm.pm[s][tid]);
            for (int s = 0; s < nsplit; ++s) {
                const float f = sm.pm[s][tid] == -INFINITY ? 0.f : ex2(sm.pm[s][tid] - top);  // no key in the share
                sm.f[s][tid] = f;
                sum += f * sm.pl[s][tid];
            }
            sm.pm[0][tid] = top;  // this CTA's own copies: cm and cl are still read by the peers
            sm.pl[0][tid] = sum;
            sm.inv[tid] = top > -INFINITY ? 1.f / sum : 0.f;
        }
        __syncthreads();
    } else {
        if (MOD) last = sm.cref;
        __syncthreads();
    }
    const int todo = min(C::kRows, rows - r0) * (D / 4);
    for (int x = split * kThreads + tid; x < todo; x += nsplit * kThreads) {
        const int r = x / (D / 4), d = x % (D / 4) * 4, row = r0 + r;
        const int tok = row / A.G, head = h * A.G + row - tok * A.G;
        float4 o;
        if (nsplit == 1) {
            o = *reinterpret_cast<const float4*>(&sm.joined[r][d]);
        } else {
            o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s) {
                if (s >= nsplit) break;
                const float4 v = peer_float4(&sm.joined[r][d], s);
                const float f = sm.f[s][r];
                o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
            }
        }
        const float inv = sm.inv[r];
        o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
        uint2 w;
        if (bf16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
            w = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        } else {
            w = make_uint2(pack_half(o.x, o.y), pack_half(o.z, o.w));
        }
        *reinterpret_cast<uint2*>(A.o + b * A.o_batch + tok * A.o_token + head * A.o_head + d) = w;
        if (d == 0) {
            const float top = nsplit == 1 ? sm.cm[r] : sm.pm[0][r], sum = nsplit == 1 ? sm.cl[r] : sm.pl[0][r];
            float e = -INFINITY;
            if (top > -INFINITY) {
                e = (top + lg2(sum)) * kLn2;
                if (MOD && A.slopes) e -= __ldg(A.slopes + head) * (float)(qpos0 + tok - last);
            }
            A.lse[((size_t)b * A.Tq + tok) * A.H * A.G + head] = e;
        }
    }
    if (nsplit > 1) cluster_sync();  // no CTA may exit while a peer reads its shared memory
}

// The shares of a selection: as many as fill the GPU in one wave, at most 8 (the portable
// cluster size), and no share below two tiles a warp.
int plan_splits(int64_t jobs, int64_t tiles, int slots) {
    const int64_t n = std::min((int64_t)slots / (jobs > 0 ? jobs : 1), tiles / (2 * kWarps));
    return (int)(n < 1 ? 1 : n > kMaxSplit ? kMaxSplit : n);
}

template <int D, int NT, bool MOD>
cudaError_t launch(cudaStream_t stream, bool bf16, const PageAttention& a, int num_sms) {
    using C = Config<D, NT>;
    const auto kernel = attend_pages_kernel<D, NT, MOD>;
    constexpr int smem = sizeof(Smem<D, NT>);
    static_assert(smem * C::kCtas <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> done{0};  // devices on which the kernel may use this much shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(done.load() >> dev & 1)) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
        if (dev < 64) done.fetch_or(1ull << dev);
    }
    const int row_tiles = (a.G * a.Tq + C::kRows - 1) / C::kRows;
    const int64_t jobs = (int64_t)a.B * a.H * row_tiles;
    const int nsplit = plan_splits(jobs, (int64_t)a.k * a.tiles, num_sms * C::kCtas);
    if (jobs * nsplit > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(jobs * nsplit));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)nsplit;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, nsplit, row_tiles, bf16);
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
