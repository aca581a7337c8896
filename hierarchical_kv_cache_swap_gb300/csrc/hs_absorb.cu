// hs_absorb.cu -- the two products that put latent attention into its absorbed form. A head's key is
// U c (128 x 512 times the latent c) beside the rotary key, so <q, U c> = <U^T q, c>: the queries take
// U over once (hs_absorb_queries, which rotates their other 64 values on the way into the rows that
// hs_attend reads), and what hs_attend gives, a sum of latents, becomes the head's output by W
// (hs_expand_outputs).
//
// Both are a batch of products over the heads, [tokens x 128][128 x 512] and [tokens x 512][512 x 128],
// with the few tokens of a decode step: memory traffic bounds them, the matrices (128 KB a head each) at
// few tokens, the rows at many, and at the smallest calls the chain from launch to store. The matrices
// are the products' rows, so that an instruction of 128 rows wastes nothing on the few tokens, which are
// its columns (tcgen05, bf16 operands, f32 sums). Measured on one GB300 (us, in a graph, with L2 cold
// where "cold"; in brackets the bytes at a copy's rate):
//   tokens x heads   1 x 128     64 x 128   256 x 128   256 x 128 cold   512 x 128 cold   37 x 20
//   queries          4.0 (2.5)   5.4 (4.3)  13.9 (9.9)  18.5 (9.9)       31.6 (17.3)      2.9
//   outputs          4.6 (2.5)   7.3 (5.3)  17.9 (13.6) 22.8 (13.6)      36.0 (24.8)      3.2
// Cold, DRAM is at 20 % (queries) and 44 % (outputs) of its peak: what is left is the time of a CTA's
// chain of copy, product and store, of which an SM has four (one) at once. CTAs of the queries that
// loop over tiles of tokens with two under way were slower (21.6 us for 256 tokens, cold), and so were
// tiles of 128 tokens (20.1 warm).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hs_latent.h"
#include "hs_launch.h"
#include "hs_once.h"
#include "hs_tc.h"

namespace hs {
namespace {

constexpr int kThreads = 256;  // of the kernel for few tokens

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>  // all groups of copies but the last LEFT have landed
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte unit u of row r in rows of 128 bytes: eight rows' units lie in different banks.
__device__ __forceinline__ uint32_t at(int r, int u) { return (uint32_t)(r * 8 + (u ^ (r & 7))) * 16; }

// ---------------------------------------------------------------- queries
// A CTA takes 128 latent dimensions (the product's rows, lanes of tensor memory) of a head and NT tokens
// (its columns): one copy brings the piece of the matrix (read across its rows: they are the product's
// inner dimension), one the tokens, and eight instructions multiply them. Meanwhile four warps rotate
// every fourth token's other values. They then bring the columns into rows of tokens in shared memory,
// neighbouring lanes exchanging a value of two columns, and one copy writes these. Several CTAs of an SM
// overlap.
constexpr int kPieces = kLatent / 128, kAbsorbThreads = 160;

struct AbsorbSmem {  // beyond the operands
    uint64_t landed, done, over;  // over: nothing is under way any more, whatever happened
    uint32_t tmem;
    volatile int abort;
};
template <int NT>
constexpr uint32_t absorb_smem() { return 1024 + 32768 + NT * 256 + sizeof(AbsorbSmem); }

struct AbsorbMaps {
    CUtensorMap w, x, out;
};

template <int NT>
__global__ void __launch_bounds__(kAbsorbThreads) absorb_kernel(const HeadProduct p, const Rotation rot,
                                                                const __grid_constant__ AbsorbMaps maps) {
    constexpr uint32_t kCols = NT < 32 ? 32 : NT;  // of tensor memory
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    AbsorbSmem* const sm = reinterpret_cast<AbsorbSmem*>(base + 32768 + NT * 256);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, piece = blockIdx.x, h = blockIdx.y;
    const int64_t t0 = (int64_t)blockIdx.z * NT, pitch = (int64_t)p.heads * (kLatent + kRope);
    uint16_t* const out = p.out + (int64_t)h * (kLatent + kRope);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 4) {
        if (lane == 0) {
            bar_init(&sm->landed, 1);
            bar_init(&sm->done, 1);
            bar_init(&sm->over, 1);
            sm->abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            bar_expect_tx(&sm->landed, 32768 + NT * 256);
            tma_load_4d(su32(base), &maps.w, 0, 0, 2 * piece, h, &sm->landed);
            if (!p.waits.stall) tma_load_4d(su32(base) + 32768, &maps.x, 0, (int)t0, 0, h, &sm->landed);
        }
        __syncwarp();
        tmem_alloc<kCols>(&sm->tmem);
    }
    // warp w rotates every 16th token: its pairs, and where they are, are loaded while the operands come
    constexpr int kTurns = NT / (4 * kPieces);
    const int first = rot.halves ? lane : 2 * lane, second = rot.halves ? lane + 32 : 2 * lane + 1;
    auto token = [&](int i) { return t0 + (i * 4 + warp) * kPieces + piece; };
    uint32_t x[kTurns], y[kTurns], mine = 0;
    int32_t pos[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        if (warp == 4 || token(i) >= p.n) continue;
        mine |= 1u << i;
        const uint16_t* const r = (const uint16_t*)p.x + token(i) * p.x_token + h * p.x_head + kHeadDim;
        x[i] = r[first];
        y[i] = r[second];
        pos[i] = rot.table ? rot.positions[token(i)] : 0;
    }
    fence_before();
    __syncthreads();
    fence_after();
    // the cosines and sines of the rotations' positions: none, and zeros, where there is no row
    float c[kTurns], s[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        c[i] = s[i] = 0.f;
        if (!rot.table || !(mine >> i & 1)) continue;
        if (pos[i] >= 0 && pos[i] < rot.rows) {
            c[i] = rot.table[(int64_t)pos[i] * kRope + lane];
            s[i] = rot.table[(int64_t)pos[i] * kRope + 32 + lane];
        } else {
            x[i] = y[i] = 0;
            if (pos[i] >= 0 && lane == 0 && h == 0 && p.status) atomicOr(p.status, 1u /* HS_STATUS_RANGE */);
        }
    }
    const uint32_t tmem = sm->tmem;
    if (warp == 4) {
        const bool ok = __all_sync(0xffffffffu, bar_wait(&sm->landed, 0, &sm->abort, p.waits.ns));
        fence_after();
        if (ok && elect_one()) {
            constexpr uint32_t id = mma_idesc(true, 128, NT, 0) | 1u << 15;  // A across its rows
            const uint32_t a = smem_desc(su32(base), 16384), b = smem_desc(su32(base) + 32768, 16);
#pragma unroll
            for (int k = 0; k < 8; ++k) mma_ss(tmem, a + 128 * k, b + NT * 8 * (k >> 2) + 2 * (k & 3), id, k ? 1u : 0u);
            mma_commit(&sm->done);
            mma_commit(&sm->over);
        }
        __syncwarp();
        if (__builtin_expect(!ok, 0)) {  // no copy lands after the CTA's end
            bar_drain(&sm->landed, 0, p.waits.drain);
            if (lane == 0) bar_arrive(&sm->over);
        }
    }
    if (warp < 4) {  // the rotations: a warp a token, a lane a pair
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            if (!(mine >> i & 1)) continue;
            float2 v = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16));
            if (rot.table) v = turn(v.x, v.y, c[i], s[i]);
            uint16_t* const o = out + token(i) * pitch + kLatent;
            const uint32_t both = pack<true>(v.x, v.y);
            if (rot.halves) {
                o[first] = (uint16_t)both;
                o[second] = (uint16_t)(both >> 16);
            } else {
                reinterpret_cast<uint32_t*>(o)[lane] = both;
            }
        }
    }
    if (warp < 4) {
        const bool ok = __all_sync(0xffffffffu, bar_wait(&sm->done, 0, &sm->abort, p.waits.ns));
        fence_after();
        if (__builtin_expect(!ok, 0)) {  // the operands' place is written below: not while copies or products use it
            bar_drain(&sm->over, 0, 4 * p.waits.drain);  // (after the issuing warp's wait and its drain)
            if (lane == 0 && p.status) atomicOr(p.status, 8u /* HS_STATUS_TIMEOUT */);
            __syncwarp();
        }
        const int odd = lane & 1, unit = (warp & 1) * 4 + (lane >> 3), byte = (lane & 6) * 2;  // of the 128-byte row of 64 dimensions
        uint8_t* const to = base + (warp >> 1) * NT * 128 + byte;
#pragma unroll
        for (int c = 0; c < NT; c += 32) {
            uint32_t v[32];
            tmem_load32(v, tmem + ((uint32_t)(warp * 32) << 16) + c);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32 && c + j < NT; j += 2) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                const float x = __uint_as_float(odd ? other : v[j]), y = __uint_as_float(odd ? v[j + 1] : other);
                const int t = c + j + odd;
                *reinterpret_cast<uint32_t*>(to + t * 128 + ((unit ^ (t & 7)) << 4)) = ok ? pack<true>(x, y) : 0x7FFF7FFFu;
            }
        }
        fence_async_smem();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (tid == 0) tma_store_4d(&maps.out, 0, (int)t0, 2 * piece, h, su32(base));
        __syncwarp();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    fence_before();
    __syncthreads();
    if (warp == 4) {
        fence_after();
        tmem_free<kCols>(tmem);
    }
}

// ---------------------------------------------------------------- outputs
// The f32 rows are sums that have not been rounded yet, and the products take each value as two bf16, its upper
// half and the rest, rounded: to within 2^-15 of it. (One bf16 each, 2^-8 of them at most, made the
// results' error against 64 bits 0.0024 of them, where their own rounding alone makes it 0.0017; it took 15.8
// us instead of 18.0 for 256 tokens of 128 heads, 3.0 instead of 3.2 for 37 of 20.)
__device__ __forceinline__ void split(float x, float y, uint32_t& upper, uint32_t& rest) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    upper = __byte_perm(a, b, 0x7632);
    // (an infinity has no rest; a NaN's is one)
    rest = pack<true>(fabsf(x) == INFINITY ? 0.f : x - __uint_as_float(a & 0xFFFF0000u), fabsf(y) == INFINITY ? 0.f : y - __uint_as_float(b & 0xFFFF0000u));
}

// Few tokens of few heads: a CTA takes 32 output dimensions and 16 tokens, all copies under way at once,
// eight steps of 64 latent dimensions. Its eight warps take a share of 16 latent dimensions each of two
// steps, so that a value is split once, and their sums are added up in the warps' order (mma.sync
// m16n8k16, which has no set-up to wait for).
constexpr int kFewTokens = 16, kFewDims = 32, kSteps = kLatent / 64, kShares = 8;
constexpr uint32_t kStepW = kFewDims * 128, kStepX = kFewTokens * 256, kStep = kStepW + kStepX;  // rows of 64 bf16, of 64 f32
constexpr uint32_t kFewSmem = kSteps * kStep;

template <int S>
__device__ __forceinline__ void steps_landed(int s) {  // steps up to s, of which each is a group of copies
    if constexpr (S < kSteps) {
        if (s == S) copies_landed<kSteps - 1 - S>();
        else steps_landed<S + 1>(s);
    }
}

__global__ void __launch_bounds__(kThreads) expand_few_kernel(const HeadProduct p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, e0 = blockIdx.x * kFewDims, h = blockIdx.y;
    const int64_t t0 = (int64_t)blockIdx.z * kFewTokens, pitch = (int64_t)p.heads * kHeadDim;
    const float* const in = (const float*)p.x + h * p.x_head;
    const uint16_t* const mat = p.w + h * p.w_head + e0 * p.w_row;
    uint16_t* const out = p.out + (int64_t)h * kHeadDim + e0 + t0 * pitch;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // 16-byte unit u of row t of x lies at u ^ 2 (t % 8): the eight rows of a fragment in different banks
    for (int s = 0; s < kSteps; ++s) {
        const uint32_t wa = su32(smem) + s * kStep, xa = wa + kStepW;
        copy16(wa + at(tid >> 3, tid & 7), mat + (tid >> 3) * p.w_row + 64 * s + 8 * (tid & 7), true);
        const int t = tid >> 4, u = tid & 15;
        const bool there = t0 + t < p.n;
        copy16(xa + t * 256 + ((u ^ (t & 7) << 1) << 4), in + (there ? t0 + t : 0) * p.x_token + 64 * s + 4 * u, there);
        copies_end();
    }
    float acc[2][4][4] = {};  // of the upper halves and of the rests, eight output dimensions each
    for (int i = 0; i < kSteps / 2; ++i) {
        steps_landed<0>(2 * i + 1);
        __syncthreads();
        const uint8_t* const w = smem + (2 * i + (warp >> 2)) * kStep;
        const uint8_t* const x = w + kStepW;
        const int share = warp & 3;  // of the step's
        uint32_t a[2][4], b[2][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // rows g and g + 8, columns 2 c and 2 c + 8 of the share's 16
            const int t = (lane >> 2) + 8 * (r & 1), u = 4 * share + 2 * (r >> 1) + ((lane & 3) >> 1);
            const float2 v = *reinterpret_cast<const float2*>(x + t * 256 + ((u ^ (t & 7) << 1) << 4) + 8 * (lane & 1));
            split(v.x, v.y, a[0][r], a[1][r]);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) ldsm(b[n], su32(w) + at(16 * n + (lane & 7) + ((lane >> 4) << 3), 2 * share + ((lane >> 3) & 1)));
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int n = 0; n < 4; ++n) mma(acc[part][n], a[part], b[n >> 1][2 * (n & 1)], b[n >> 1][2 * (n & 1) + 1]);
    }
    __syncthreads();  // the operands' place becomes the shares'
    float* const sums = reinterpret_cast<float*>(smem);  // [kShares][kFewTokens][kFewDims]
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2*>(sums + (warp * kFewTokens + 8 * r + (lane >> 2)) * kFewDims + 8 * n + 2 * (lane & 3)) =
                make_float2(acc[0][n][2 * r] + acc[1][n][2 * r], acc[0][n][2 * r + 1] + acc[1][n][2 * r + 1]);
    __syncthreads();
    const int t = tid >> 4, e = 2 * (tid & 15);  // a thread two dimensions of a token
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kShares; ++s) {
        const float2 y = *reinterpret_cast<const float2*>(sums + (s * kFewTokens + t) * kFewDims + e);
        v = make_float2(v.x + y.x, v.y + y.y);
    }
    if (t0 + t < p.n) *reinterpret_cast<uint32_t*>(out + t * pitch + e) = pack<true>(v.x, v.y);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Many tokens: a CTA brings its head's whole matrix (128 output dimensions: the product's rows) into tensor
// memory, 256 columns, and takes tiles of 32 tokens, each by one of two groups of eight warps: they load a
// tile's f32 rows straight into registers, split them into shared memory (64 rows: the tokens' upper halves,
// then their rests: the product's columns), and load the next ones while one thread multiplies and all write
// the sums of the two halves' columns, two tokens at a time as above. The two groups' tiles keep 128 KB of
// loads under way, which is what it takes to draw an SM's share of the memory's rate. The matrix comes by way
// of the tiles' place, before the first ones: 1.1 us a CTA, but then both halves of the rows have room there
// (with the matrix in shared memory and tiles in four stages 512 tokens of 128 heads took 46 us instead of 36).
constexpr int kTokens = 32, kGroupThreads = 256, kManyThreads = 2 * kGroupThreads, kCols = 2 * kTokens;
struct ExpandSmem {  // beyond the operands
    uint64_t landed[4], done[2], over[2];  // landed: a quarter of the matrix; over: a tile's products have ended, or there are none, whatever happened
    uint32_t tmem;
    volatile int abort;
};
constexpr uint32_t kMatrix = kHeadDim * kLatent * 2, kTile64 = kCols * 128, kTokenTile = kLatent / 64 * kTile64;
constexpr uint32_t kManyTmem = 512, kMatrixCols = kLatent / 2;
constexpr uint32_t kManySmem = 1024 + 2 * kTokenTile + sizeof(ExpandSmem);
static_assert(kMatrix <= 2 * kTokenTile, "the matrix comes by way of the tiles' place");

__global__ void __launch_bounds__(kManyThreads, 1) expand_many_kernel(const HeadProduct p, const __grid_constant__ CUtensorMap map) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    ExpandSmem* const sm = reinterpret_cast<ExpandSmem*>(base + 2 * kTokenTile);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31, h = blockIdx.x;
    const int group = warp >> 3, tid = threadIdx.x & (kGroupThreads - 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) bar_init(&sm->landed[i], 1);
        for (int i = 0; i < 2; ++i) bar_init(&sm->done[i], 1), bar_init(&sm->over[i], 1);
        sm->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int c = 0; c < 4; ++c) {
            bar_expect_tx(&sm->landed[c], kMatrix / 4);
            if (!p.waits.stall || c > 0) tma_load_4d(su32(base) + c * (kMatrix / 4), &map, 0, 0, 2 * c, h, &sm->landed[c]);
        }
    }
    if (warp == 0) tmem_alloc<kManyTmem>(&sm->tmem);
    // unit u (8 values) of the group's tile: of token u / 64, dimensions 8 (u % 64) on
    const float* const in = (const float*)p.x + h * p.x_head;
    const int64_t step = (int64_t)gridDim.y * 2 * kTokens, pitch = (int64_t)p.heads * kHeadDim;
    constexpr int kUnits = kTokens * kLatent / 8 / kGroupThreads;  // of a thread
    uint8_t* const x = base + group * kTokenTile;
    float4 v[2 * kUnits];
    uint4 upper[kUnits], rest[kUnits];
    auto fetch = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = i * kGroupThreads + tid;
            const int64_t t = t0 + (u >> 6);
            if (t < p.n) {
                const float4* const r = reinterpret_cast<const float4*>(in + t * p.x_token) + 2 * (u & 63);
                v[2 * i] = r[0];
                v[2 * i + 1] = r[1];
            } else {
                v[2 * i] = v[2 * i + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    };
    auto halve = [&] {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            split(v[2 * i].x, v[2 * i].y, upper[i].x, rest[i].x);
            split(v[2 * i].z, v[2 * i].w, upper[i].y, rest[i].y);
            split(v[2 * i + 1].x, v[2 * i + 1].y, upper[i].z, rest[i].z);
            split(v[2 * i + 1].z, v[2 * i + 1].w, upper[i].w, rest[i].w);
        }
    };
    int64_t t0 = ((int64_t)blockIdx.y * 2 + group) * kTokens;
    fetch(t0);
    fence_before();
    __syncthreads();
    fence_after();
    // The matrix, from rows of 128 swizzled bytes: a lane a row, warps w, w + 4, w + 8 and w + 12 a quarter each.
    const uint32_t matrix = sm->tmem, lanes = (uint32_t)((warp & 3) * 32) << 16, cols = matrix + kMatrixCols + group * kCols;
    const bool landed = __all_sync(0xffffffffu, bar_wait(&sm->landed[warp >> 2], 0, &sm->abort, p.waits.ns));
    if (__builtin_expect(!landed, 0)) bar_drain(&sm->landed[warp >> 2], 0, p.waits.drain);  // the tiles' place is written below
#pragma unroll 1
    for (int c = 2 * (warp >> 2); c < 2 * (warp >> 2) + 2; ++c) {
        const int row = (warp & 3) * 32 + lane;
        const uint4* const from = reinterpret_cast<const uint4*>(base + c * (kHeadDim * 128) + row * 128);
        uint32_t r[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint4 w = from[u ^ (row & 7)];
            r[4 * u] = w.x, r[4 * u + 1] = w.y, r[4 * u + 2] = w.z, r[4 * u + 3] = w.w;
        }
        tmem_store32(matrix + lanes + 32 * c, r);
    }
    tmem_wait_st();
    fence_before();
    __syncthreads();
    fence_after();
    bool ok = !sm->abort;  // one for all warps: who set it did before they met
    for (int k = 0; t0 < p.n; t0 += step, ++k) {
        halve();
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = i * kGroupThreads + tid, t = u >> 6, c = u & 63;  // a column of 64 dimensions after the other
            uint8_t* const to = x + (c >> 3) * kTile64 + t * 128 + (((c & 7) ^ (t & 7)) << 4);
            *reinterpret_cast<uint4*>(to) = upper[i];
            *reinterpret_cast<uint4*>(to + kTokens * 128) = rest[i];
        }
        fence_async_smem();
        fence_before();
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroupThreads) : "memory");
        if (t0 + step < p.n) fetch(t0 + step);
        if ((warp & 7) == 0) {
            fence_after();
            if (ok && elect_one()) {
                constexpr uint32_t id = mma_idesc(true, kHeadDim, kCols, 0);
                const uint32_t b = smem_desc(su32(x), 16);
#pragma unroll
                for (int s = 0; s < kLatent / 16; ++s) mma_ts(cols, matrix + 8 * s, b + (s >> 2) * (kTile64 / 16) + 2 * (s & 3), id, s ? 1u : 0u);
                mma_commit(&sm->done[group]);
                mma_commit(&sm->over[group]);
            }
            if (__builtin_expect(!ok, 0) && lane == 0) bar_arrive(&sm->over[group]);
            __syncwarp();
        }
        ok = __all_sync(0xffffffffu, ok && bar_wait(&sm->done[group], k & 1, &sm->abort, p.waits.ns));
        if (__builtin_expect(!ok, 0)) {  // the tile's place is not written again, nor the columns freed, under its products
            bar_drain(&sm->over[group], k & 1, 4 * p.waits.drain);
            if (lane == 0 && p.status) atomicOr(p.status, 8u /* HS_STATUS_TIMEOUT */);
            __syncwarp();
        }
        fence_after();
        // warps w and w + 4 share 32 output dimensions: half of the tokens each
        uint32_t both[2][16], d[16];
        const int half = (warp >> 2) & 1, odd = lane & 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) tmem_load16(both[i], cols + lanes + i * kTokens + 16 * half);
        tmem_wait_ld();
        fence_before();
#pragma unroll
        for (int j = 0; j < 16; ++j) d[j] = __float_as_uint(__uint_as_float(both[0][j]) + __uint_as_float(both[1][j]));
        uint16_t* const to = p.out + h * kHeadDim + (warp & 3) * 32 + (lane & ~1);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? d[j] : d[j + 1], 1);
            const float lo = __uint_as_float(odd ? other : d[j]), hi = __uint_as_float(odd ? d[j + 1] : other);
            const int64_t t = t0 + 16 * half + j + odd;
            if (t < p.n) *reinterpret_cast<uint32_t*>(to + t * pitch) = ok ? pack<true>(lo, hi) : 0x7FFF7FFFu;
        }
        // after an abort, too: warps may differ in whether a wait ran out, and the others come here
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroupThreads) : "memory");  // all have read the columns
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        tmem_free<kManyTmem>(sm->tmem);
    }
}

struct Ready {};
template <class K>
cudaError_t allow(K* kernel, uint32_t smem) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); }

// The kernels' shared memory, allowed once on each device.
cudaError_t set_up() {
    static PerDevice<Ready> devices;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device >= PerDevice<Ready>::kDevices) return cudaErrorInvalidDevice;
    const Ready* ready;
    return (cudaError_t)devices.get(device, [](Ready*) {
        cudaError_t x = allow(absorb_kernel<16>, absorb_smem<16>());
        if (x == cudaSuccess) x = allow(absorb_kernel<64>, absorb_smem<64>());
        if (x == cudaSuccess) x = allow(expand_few_kernel, kFewSmem);
        if (x == cudaSuccess) x = allow(expand_many_kernel, kManySmem);
        return (int)x;
    }, &ready);
}

int64_t tiles(int64_t n, int of) { return (n + of - 1) / of; }

}  // namespace

cudaError_t launch_absorb_queries(cudaStream_t stream, const HeadProduct& p, const Rotation& rot, int num_sms) {
    if (p.n == 0 || p.heads == 0) return cudaSuccess;
    cudaError_t e = set_up();
    if (e != cudaSuccess) return e;
    // 16 tokens a CTA while all CTAs fit the SMs at once, 64 beyond (37 tokens of 20 heads: 3.0 us against
    // 3.6; 64 of 128 heads: 10.6 against 6.2)
    const int nt = 4 * tiles(p.n, 16) * p.heads <= 4 * (int64_t)num_sms ? 16 : 64;
    AbsorbMaps maps;
    if (!encode_columns(&maps.w, true, p.w, kHeadDim, kLatent / 64, p.heads, p.w_row, p.heads > 1 ? p.w_head : kHeadDim * kLatent, kHeadDim, 2) ||
        !encode_columns(&maps.x, true, (const uint16_t*)p.x, p.n, kHeadDim / 64, p.heads, p.n > 1 ? p.x_token : kHeadDim, p.heads > 1 ? p.x_head : kHeadDim, nt, 2) ||
        !encode_columns(&maps.out, true, p.out, p.n, (kLatent + kRope) / 64, p.heads, (int64_t)p.heads * (kLatent + kRope), kLatent + kRope, nt, 2))
        return cudaErrorInvalidValue;
    const dim3 grid(kPieces, p.heads, (unsigned)tiles(p.n, nt));
    if (nt == 16) return launch_dependent(stream, grid, kAbsorbThreads, absorb_smem<16>(), absorb_kernel<16>, p, rot, maps);
    return launch_dependent(stream, grid, kAbsorbThreads, absorb_smem<64>(), absorb_kernel<64>, p, rot, maps);
}

cudaError_t launch_expand_outputs(cudaStream_t stream, const HeadProduct& p, int num_sms) {
    if (p.n == 0 || p.heads == 0) return cudaSuccess;
    cudaError_t e = set_up();
    if (e != cudaSuccess) return e;
    // few tokens of few heads: pieces of 32 output dimensions of 16 tokens, while all CTAs run at once, three an
    // SM. us of this kernel and of the other, in a graph, by CTAs (152 SMs): 320 (80 tokens of 16 heads) 3.9 and
    // 6.7, 384 (16 of 96) 4.0 and 5.0, 512 (128 of 16) 4.9 and 6.8, 512 (16 of 128) 4.9 and 5.0, 512 (1 of 128)
    // 5.0 and 4.6, 768 (48 of 64) 6.6 and 6.6, 1024 (256 of 16) 7.8 and 6.9, 1536 (48 of 128) 11.2 and 6.9
    const dim3 few(kHeadDim / kFewDims, p.heads, (unsigned)tiles(p.n, kFewTokens));
    if ((int64_t)few.x * few.y * few.z <= 3 * (int64_t)num_sms) return launch_dependent(stream, few, kThreads, kFewSmem, expand_few_kernel, p);
    CUtensorMap map;
    if (!encode_columns(&map, true, p.w, kHeadDim, kLatent / 64, p.heads, p.w_row, p.heads > 1 ? p.w_head : kHeadDim * kLatent, kHeadDim, 2)) return cudaErrorInvalidValue;
    // a head's CTAs are as many as run at once with the other heads': a second round of them would read the
    // matrices again (256 tokens of 128 heads, cold: 20.5 us, 22.9 in two). More heads than SMs take two
    // all the same (64 tokens of 160 heads 13.2 us, of 128 heads 7.2), 80 heads leave half of the SMs idle
    const int64_t most = p.heads < num_sms ? num_sms / p.heads : 1, t = tiles(p.n, 2 * kTokens);
    return launch_dependent(stream, dim3(p.heads, (unsigned)(t < most ? t : most)), kManyThreads, kManySmem, expand_many_kernel, p, map);
}

}  // namespace hs
