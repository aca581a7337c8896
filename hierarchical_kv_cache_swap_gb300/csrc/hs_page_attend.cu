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

#include <atomic>

#include "hs_page.h"

namespace hs {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kListTiles = 1024;       // tiles listed at a time
constexpr float kRescale = 8.f;        // a row's reference maximum moves when exceeded by 2^8
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

template <int D, int NT>
struct Config {
    static constexpr int kChunk = 18 * D;           // bytes of a tile of one head
    static constexpr int kRows = 8 * NT;            // query rows of a CTA
    static constexpr int kSteps = D / 16;
    static constexpr int kCtas = NT * D <= 128 ? 2 : 1;  // CTAs an SM: registers
    static constexpr int kStages = D == 64 ? 6 : D == 128 ? 4 : 4;
    static constexpr int kRing = kWarps * kStages * kChunk;
    static constexpr int kPart = kWarps * kRows * D * 4;  // the warps' outputs, over the ring
    static constexpr int kSpace = kRing > kPart ? kRing : kPart;
};

template <int D, int NT>
struct Smem {
    using C = Config<D, NT>;
    alignas(128) uint8_t space[C::kSpace];
    alignas(16) uint16_t q[C::kRows][D + 8];  // the rows as halves, scaled
    float joined[C::kRows][D];                // this CTA's output, relative to its maxima
    float m[kWarps][C::kRows], l[kWarps][C::kRows];
    float cm[C::kRows], cl[C::kRows];         // this CTA's maxima and sums
    float qscale[C::kRows];
    uint64_t bar[kWarps][C::kStages];
    int2 list[kListTiles];                    // unit (slot * tiles + tile), position | partial
    int count[kListTiles / 32];
    int kref[kWarps];
    int ref;                                  // position that biases are relative to
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
__device__ __forceinline__ uint32_t scale2(uint32_t u) { return u << 7 | u << 23; }  // (s, s) of scale byte u
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
    int64_t job = blockIdx.x / nsplit;
    const int split = (int)(blockIdx.x - job * nsplit);  // = the rank in the cluster
    const int rt = (int)(job % row_tiles);
    job /= row_tiles;
    const int h = (int)(job % A.H), b = (int)(job / A.H);
    const int rows = A.G * A.Tq, r0 = rt * C::kRows;

    if (tid < kWarps * C::kStages) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(su32(&sm.bar[0][0] + tid)) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    // the request's mask: row token t sees p <= length - Tq + t and (p >= start or p < prefix)
    const int length = __ldg(A.lengths + b);
    const int start = A.start ? __ldg(A.start + b) : 0;
    const int prefix = A.prefix ? __ldg(A.prefix + b) : 0;
    const int qpos0 = length - A.Tq;  // may be negative
    const int j0 = (int)((int64_t)A.k * split / nsplit), j1 = (int)((int64_t)A.k * (split + 1) / nsplit);
    const int32_t* slots = A.slots + (size_t)b * A.k;
    const int32_t* sel = A.sel + (size_t)b * A.k;
    const int ntiles = (j1 - j0) * A.tiles;  // of this CTA's share
    const uint8_t* pages = A.pages + ((size_t)b * A.S * A.tiles * A.H + h) * C::kChunk;
    const size_t unit_bytes = (size_t)A.H * C::kChunk;

    // the query rows as halves
    for (int r = warp; r < C::kRows; r += kWarps) {
        constexpr int N = D / 32;
        float x[N];
        const int row = r0 + r;
        float scale = 0.f;
        if (row < rows) {
            const int tok = row / A.G, head = h * A.G + row % A.G;
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
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) sm.q[r][lane * N + i] = __half_as_ushort(__float2half_rn(x[i]));
        // to log2 units; with a cap, to 2 log2 e s / cap
        if (lane == 0) sm.qscale[r] = MOD && A.cap > 0.f ? scale * (A.scale * (2.f * kLog2e / A.cap)) : scale * (A.scale * kLog2e);
    }
    // biases are taken relative to the last position of the share, so that far shares keep
    // their differences (the whole bias of a far key has few fraction bits left in f32)
    if (MOD) {
        int last = -1;
        for (int j = j0 + tid; j < j1; j += kThreads) {
            const int s = __ldg(slots + j), p = __ldg(sel + j);
            if (s >= 0 && s < A.S && p >= 0) {
                const int64_t e = ((int64_t)p + 1) * (A.tiles * kTile) - 1;
                if (e - (A.tiles * kTile - 1) < length) last = max(last, (int)min(e, (int64_t)length - 1));
            }
        }
        last = __reduce_max_sync(0xffffffffu, last);
        if (lane == 0) sm.kref[warp] = last;
    }
    __syncthreads();
    int ref = 0;
    if (MOD) {
        ref = sm.kref[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) ref = max(ref, sm.kref[w]);
    }

    // this lane's part of Q, and its rows' factors (rows 8 n + 2 t, + 1)
    uint32_t qf[NT][C::kSteps][2];
    float qs[NT][2], slope[NT][2];
    int qpos[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < C::kSteps; ++i) {
            const uint2 w = *reinterpret_cast<const uint2*>(&sm.q[8 * n + g][t * (D / 4) + 4 * i]);
            qf[n][i][0] = w.x;
            qf[n][i][1] = w.y;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int row = min(r0 + 8 * n + 2 * t + c, rows - 1);
            qs[n][c] = sm.qscale[8 * n + 2 * t + c];
            qpos[n][c] = qpos0 + row / A.G;
            slope[n][c] = MOD && A.slopes ? __ldg(A.slopes + h * A.G + row % A.G) * kLog2e : 0.f;
        }
    }
    const float cap2 = A.cap * kLog2e;

    float acc[C::kSteps][NT][4];  // O^T: dims g D/8 + 2 i, + 1 (c = 0, 1 and 2, 3), rows 8 n + 2 t, + 1
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

    uint8_t* ring = sm.space + warp * (C::kStages * C::kChunk);
    uint64_t* bar = sm.bar[warp];
    uint32_t fill = 0, use = 0;  // copies issued and waited for by this warp
    bool ok = true;

    for (int base = 0; base < ntiles; base += kListTiles) {
        // the share's next live tiles, in order
        const int here = min(kListTiles, ntiles - base);
        int2 mine[kListTiles / kThreads];
        uint32_t live[kListTiles / kThreads];
#pragma unroll
        for (int i = 0; i < kListTiles / kThreads; ++i) {
            const int x = i * kThreads + tid;
            bool is = false;
            if (x < here) {
                const int j = (base + x) / A.tiles, tile = base + x - j * A.tiles;
                const int s = __ldg(slots + j0 + j), p = __ldg(sel + j0 + j);
                const int64_t at = (int64_t)p * (A.tiles * kTile) + tile * kTile;
                if (s >= A.S && A.status) atomicOr(A.status, 1u /* HS_STATUS_RANGE */);
                if (s >= 0 && s < A.S && p >= 0 && at < length) {
                    const int pos = (int)at, end = pos + (kTile - 1);
                    const bool in = !A.start || end >= start || pos < prefix;
                    const bool full = end <= qpos0 && (!A.start || pos >= start || end < prefix);
                    is = in;
                    mine[i] = make_int2(s * A.tiles + tile, pos | (full ? 0 : 1));
                }
            }
            live[i] = __ballot_sync(0xffffffffu, is);
            if (lane == 0) sm.count[i * kWarps + warp] = __popc(live[i]);
        }
        __syncthreads();
        int total;
        {
            const int c = sm.count[lane];  // 32 counts, in the tiles' order
            int sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            total = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
            for (int i = 0; i < kListTiles / kThreads; ++i) {
                const int before = __shfl_sync(0xffffffffu, sum - c, i * kWarps + warp);
                if (live[i] >> lane & 1u) sm.list[before + __popc(live[i] & ((1u << lane) - 1u))] = mine[i];
            }
        }
        __syncthreads();

        auto issue = [&](int x) {  // the copy of listed tile x
            if (lane == 0) {
                const int st = fill % C::kStages;
                copy_in(ring + st * C::kChunk, pages + (size_t)sm.list[x].x * unit_bytes, C::kChunk, &bar[st]);
            }
            ++fill;
        };
        // after a wait that ran out the warp takes part in the barriers only
#pragma unroll 1
        for (int i = 0; i < C::kStages; ++i)
            if (ok && warp + i * kWarps < total) issue(warp + i * kWarps);
#pragma unroll 1
        for (int x = warp; ok && x < total; x += kWarps) {
            const int st = use % C::kStages;
            const uint8_t* tile = ring + st * C::kChunk;
            if (!__all_sync(0xffffffffu, bar_wait(&bar[st], (use / C::kStages) & 1u, deadline))) {
                ok = false;
                break;
            }
            ++use;
            const int word = sm.list[x].y;
            const int pos = word & ~15;
            const bool partial = word & 1;

            // ---------------- S^T = K Q^T
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            {
                uint32_t kw[2][D / 32];  // D/8 bytes of keys g and g + 8
                uint32_t ku[2];          // their D/64 scale bytes
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint8_t* src = tile + (g + 8 * c) * (D / 2) + t * (D / 8);
                    const uint8_t* us = tile + 8 * D + (g + 8 * c) * (D / 16) + t * (D / 64);
                    if (D == 64) {
                        const uint2 v = *reinterpret_cast<const uint2*>(src);
                        kw[c][0] = v.x; kw[c][1] = v.y;
                        ku[c] = *us;
                    } else {
#pragma unroll
                        for (int i = 0; i < D / 128; ++i) {
                            const uint4 v = reinterpret_cast<const uint4*>(src)[i];
                            kw[c][4 * i] = v.x; kw[c][4 * i + 1] = v.y; kw[c][4 * i + 2] = v.z; kw[c][4 * i + 3] = v.w;
                        }
                        ku[c] = D == 128 ? *reinterpret_cast<const uint16_t*>(us) : *reinterpret_cast<const uint32_t*>(us);
                    }
                }
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {  // a word: 8 dims, two steps
                    const uint32_t sc0 = scale2(ku[0] >> (8 * (w / 2)) & 0xFFu), sc1 = scale2(ku[1] >> (8 * (w / 2)) & 0xFFu);
                    uint32_t a[4], c[4];
                    decode_word(kw[0][w], a);
                    decode_word(kw[1][w], c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i] = mul2(a[i], sc0);
                        c[i] = mul2(c[i], sc1);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma(s[n], a[0], c[0], a[1], c[1], qf[n][2 * w][0], qf[n][2 * w][1]);
                        mma(s[n], a[2], c[2], a[3], c[3], qf[n][2 * w + 1][0], qf[n][2 * w + 1][1]);
                    }
                }
            }

            // ---------------- scores in log2 units, masked; s[n][c + 2 k]: row c, key g + 8 k
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float y = s[n][c] * qs[n][c & 1];
                    if (MOD) {
                        if (A.cap > 0.f) y = cap2 * tanh_of(y);
                        y -= slope[n][c & 1] * (float)(ref - (pos + g + 8 * (c >> 1)));
                    }
                    s[n][c] = y;
                }
            bool more = false;
            if (partial) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int p = pos + g + 8 * k;
                    const bool in = !A.start || p >= start || p < prefix;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (!in || p > qpos[n][c]) s[n][c + 2 * k] = -INFINITY;
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) more |= !(s[n][c] <= m[n][c & 1] + kRescale);
            if (__any_sync(0xffffffffu, more)) {  // a row's maximum has grown: move every row's reference
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        // a NaN score counts as +inf here, so that the join keeps the row's NaNs
                        float top = fmaxf(s[n][c] == s[n][c] ? s[n][c] : INFINITY, s[n][c + 2] == s[n][c + 2] ? s[n][c + 2] : INFINITY);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const float now = fmaxf(m[n][c], top);
                        const float f = now > -INFINITY ? ex2(m[n][c] - now) : 1.f;
                        m[n][c] = now;
                        l[n][c] *= f;
#pragma unroll
                        for (int i = 0; i < C::kSteps; ++i) {
                            acc[i][n][c] *= f;
                            acc[i][n][c + 2] *= f;
                        }
                    }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // a row without a key yet has s = m = -inf
                    const float w = partial && s[n][c] == -INFINITY ? 0.f : ex2(s[n][c] - m[n][c & 1]);
                    l[n][c & 1] += w;
                    s[n][c] = w;
                }
                pf[n][0] = transpose8x8(pack_half(s[n][0], s[n][1]));
                pf[n][1] = transpose8x8(pack_half(s[n][2], s[n][3]));
            }

            // ---------------- O^T += V^T P
            {
                constexpr int W = D / 64;  // words of codes a token: D/8 dims
                uint32_t vw[4][W], vs[4];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int tok = 2 * t + (c & 1) + 8 * (c >> 1);
                    const uint8_t* src = tile + 9 * D + tok * (D / 2) + g * (D / 16);
                    const uint8_t* us = tile + 17 * D + tok * (D / 16);
                    if (D == 64) {
                        vw[c][0] = *reinterpret_cast<const uint32_t*>(src);
                        vs[c] = us[g >> 1];
                    } else if (D == 128) {
                        const uint2 v = *reinterpret_cast<const uint2*>(src);
                        vw[c][0] = v.x; vw[c][W - 1] = v.y;
                        vs[c] = us[g];
                    } else {
                        const uint4 v = *reinterpret_cast<const uint4*>(src);
                        vw[c][0] = v.x; vw[c][1] = v.y; vw[c][W - 2] = v.z; vw[c][W - 1] = v.w;
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
                        const int tok = 2 * t + (c & 1) + 8 * (c >> 1), p = pos + tok;
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
                                const int seen = qpos[n][c] - pos;  // the row sees tokens 0 .. seen of the tile
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
                        for (int n = 0; n < NT; ++n) mma(acc[4 * w + i][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read the stage: refill it
            if (x + C::kStages * kWarps < total) issue(x + C::kStages * kWarps);
        }
        __syncthreads();  // the list is rebuilt
    }
    if (!ok && A.status && lane == 0) atomicOr(A.status, 8u /* HS_STATUS_TIMEOUT */);
    if (!ok) {  // no copy may still be landing when the CTA exits: wait for them, bounded again
        const uint64_t by = global_ns() + kDefaultWaitNs;
        for (; use != fill; ++use) bar_wait(&bar[use % C::kStages], (use / C::kStages) & 1u, by);
    }
    __syncthreads();

    // ---------------- join the warps
    float* part = reinterpret_cast<float*>(sm.space);  // [warp][row][D]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float sum = l[n][c];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const int r = 8 * n + 2 * t + c;
            if (g == 0) {
                sm.m[warp][r] = m[n][c];
                sm.l[warp][r] = sum;
            }
            float* dst = part + ((size_t)warp * C::kRows + r) * D + g * (D / 8);
#pragma unroll
            for (int i = 0; i < C::kSteps; ++i) *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(acc[i][n][c], acc[i][n][c + 2]);
        }
    if (tid == 0) sm.ref = ref;
    __syncthreads();
    for (int x = tid; x < C::kRows * (D / 4); x += kThreads) {
        const int r = x / (D / 4), d = x % (D / 4) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.m[w][r]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (sm.m[w][r] == -INFINITY) continue;  // the warp saw no key of this row
            const float f = ex2(sm.m[w][r] - top);
            const float4 v = *reinterpret_cast<const float4*>(part + ((size_t)w * C::kRows + r) * D + d);
            sum += f * sm.l[w][r];
            o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
        }
        *reinterpret_cast<float4*>(&sm.joined[r][d]) = o;
        if (d == 0) {
            sm.cm[r] = top;
            sm.cl[r] = sum;
        }
    }
    // ---------------- join the shares, each CTA a part of the rows' elements, and write
    if (nsplit > 1) cluster_sync();
    else __syncthreads();
    int far = ref;
    if (MOD && A.slopes)
        for (int s = 0; s < nsplit; ++s) far = max(far, nsplit > 1 ? peer_int(&sm.ref, s) : ref);
    const int todo = min(C::kRows, rows - r0) * (D / 4);
    for (int x = split * kThreads + tid; x < todo; x += nsplit * kThreads) {
        const int r = x / (D / 4), d = x % (D / 4) * 4, row = r0 + r;
        const int tok = row / A.G, head = h * A.G + row % A.G;
        const float sl = MOD && A.slopes ? __ldg(A.slopes + head) * kLog2e : 0.f;
        float4 o;
        float top, sum;
        if (nsplit == 1) {
            o = *reinterpret_cast<const float4*>(&sm.joined[r][d]);
            top = sm.cm[r];
            sum = sm.cl[r];
        } else {
            top = -INFINITY;
            for (int s = 0; s < nsplit; ++s) {
                float ms = peer_float(&sm.cm[r], s);
                if (MOD && sl != 0.f) ms -= sl * (float)(far - peer_int(&sm.ref, s));
                top = fmaxf(top, ms);
            }
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            sum = 0.f;
            for (int s = 0; s < nsplit; ++s) {
                float ms = peer_float(&sm.cm[r], s);
                if (MOD && sl != 0.f) ms -= sl * (float)(far - peer_int(&sm.ref, s));
                if (ms == -INFINITY) continue;  // the share holds no key of this row
                const float f = ex2(ms - top);
                const float4 v = peer_float4(&sm.joined[r][d], s);
                sum += f * peer_float(&sm.cl[r], s);
                o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
            }
        }
        const float inv = top > -INFINITY ? 1.f / sum : 0.f;
        o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
        uint16_t* dst = A.o + b * A.o_batch + tok * A.o_token + head * A.o_head + d;
        uint2 w;
        if (bf16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
            w = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        } else {
            w = make_uint2(pack_half(o.x, o.y), pack_half(o.z, o.w));
        }
        *reinterpret_cast<uint2*>(dst) = w;
        if (d == 0) {
            float e = -INFINITY;
            if (top > -INFINITY) {
                e = (top + lg2(sum)) * kLn2;
                if (MOD && sl != 0.f) e -= __ldg(A.slopes + head) * (float)(qpos0 + tok - far);
            }
            A.lse[((size_t)b * A.Tq + tok) * A.H * A.G + head] = e;
        }
    }
    if (nsplit > 1) cluster_sync();  // no CTA may exit while a peer reads its shared memory
}

// The shares of a selection: enough CTAs to fill the GPU, at most 8 (the portable cluster),
// and no share below two tiles a warp.
int plan_splits(int64_t jobs, int64_t tiles, int ctas) {
    int n = 1;
    while (n < 8 && jobs * n < ctas && tiles / (2 * n) >= 2 * kWarps) n *= 2;
    return n;
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
