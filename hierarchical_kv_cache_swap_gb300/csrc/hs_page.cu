// hs_page.cu -- tokens quantised into 4-bit pages as they are written, and pages read back.
//
// A block is 16 consecutive dimensions of one token's K or V row of one head. It is stored
// as 16 E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign) and one scale byte u, the
// half-precision number with bits u << 7 (five exponent bits, three fraction bits). Writing
// takes a = max |x|, the scale s nearest to a / 6 (ties to the even byte, at most 10240) and
// the code nearest to x / s (ties to the even code, at most 6). Reading gives code * s: the
// code has two significant bits and the scale four, so the value has at most six and is
// exact in bf16 and in fp16, where it is always finite (6 * 10240 = 61440). A block that
// holds an infinity or a NaN gets a NaN scale and reads back as NaN.
//
// One thread makes (or reads) one block of K and the same block of V at a time: 2 x 32 bytes
// of 16-bit floats against 2 x 9 bytes of page. The lanes of a warp take the D / 16 blocks of
// a row and 512 / D consecutive tokens of one head, whose codes lie together in the page (256
// bytes, and 32 bytes of scales), so both sides move in whole 32-byte sectors. Both kernels
// are bound by memory traffic: 2 + 9/16 bytes a value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hs_page.h"

namespace hs {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t bits) {
    if (BF16) return __uint_as_float((uint32_t)bits << 16);
    return __half2float(__ushort_as_half(bits));
}

__device__ __forceinline__ float scale_value(uint32_t u) { return __half2float(__ushort_as_half((uint16_t)(u << 7))); }

// The scale byte nearest to t >= 0. In the normal range the byte is the top of t's own bits
// (re-biased), rounded to three fraction bits; below it the scales are multiples of 2^-17.
__device__ __forceinline__ uint32_t scale_byte(float t) {
    const uint32_t b = __float_as_uint(t);
    uint32_t u;
    if (t >= 6.103515625e-5f) {  // 2^-14
        u = ((b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20) - ((127 - 15) << 3);
    } else {
        u = (uint32_t)__float2int_rn(t * 131072.f);  // 2^17
    }
    return min(u, (uint32_t)kTopScale);
}

// Two values to two codes in a byte (a: low half).
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    uint32_t r;
    asm("{ .reg .b8 c; cvt.rn.satfinite.e2m1x2.f32 c, %2, %1; mov.b32 %0, {c, 0, 0, 0}; }" : "=r"(r) : "f"(a), "f"(b));
    return r;
}

// Eight codes with every negative zero made code 0.
__device__ __forceinline__ uint32_t one_zero(uint32_t w) {
    const uint32_t some = (w | w >> 1 | w >> 2) & 0x11111111u;  // magnitudes that are not zero
    return w & (0x77777777u | some << 3);
}

struct Block {
    uint32_t lo, hi;  // 16 codes
    uint32_t u;       // scale byte
};

// Sixteen 16-bit floats (w: 8 words) to a block.
template <bool BF16>
__device__ __forceinline__ Block quantise(const uint32_t (&w)[8]) {
    // the magnitudes' bits order like the magnitudes, infinities and NaNs above every number
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    const bool bad = m >= (BF16 ? 0x7F80u : 0x7C00u);
    Block r;
    r.u = bad ? 0u : scale_byte(to_float<BF16>((uint16_t)m) / 6.f);
    const float inv = r.u ? 1.f / scale_value(r.u) : 0.f;
    // x / s decides ties exactly although 1 / s is rounded: x * inv is brought to multiples of
    // 2^-13 (adding 1536 leaves 13 fraction bits), which every border between codes is. A
    // quotient on a border is off by 2^-24 relative before that and lands on it again; one that
    // is not differs from the border t s by at least one unit of x's last place, so by 2^-11
    // relative, 2^-13 at the smallest border (1/4): it stays on its side.
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = __fmaf_rn(to_float<BF16>((uint16_t)w[i]), inv, 1536.f) - 1536.f;
        const float b = __fmaf_rn(to_float<BF16>((uint16_t)(w[i] >> 16)), inv, 1536.f) - 1536.f;
        c[i] = codes2(a, b);
    }
    r.lo = one_zero(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24);
    r.hi = one_zero(c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
    if (bad) {
        r.lo = r.hi = 0;
        r.u = kBadScale;
    }
    return r;
}

__device__ __forceinline__ void load_block(uint32_t (&w)[8], const uint16_t* p) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

template <int D>
__device__ __forceinline__ void store_block(uint8_t* chunk, int row, int blk, const Block& b) {
    *reinterpret_cast<uint2*>(chunk + row * (D / 2) + 8 * blk) = make_uint2(b.lo, b.hi);
    chunk[8 * D + row * (D / 16) + blk] = (uint8_t)b.u;
}

// Where a token goes: the tile of its page (without the head's offset) in one or two places.
struct Place {
    uint8_t* a;
    uint8_t* b;  // or nullptr
    int row;     // of the tile; < 0: the token is skipped
};

struct ToPages {
    const int64_t* dest;
    uint8_t* pages;
    int64_t slots;      // token slots: num_pages * tokens
    size_t tile_bytes;  // the tiles of all pages lie one after the other
    uint32_t* status;
    __device__ __forceinline__ Place operator()(int64_t i, bool first) const {
        const int64_t d = __ldg(dest + i);
        if (d < 0) return {nullptr, nullptr, -1};
        if (d >= slots) {
            if (first && status) atomicOr(status, 1u /* HS_STATUS_RANGE */);
            return {nullptr, nullptr, -1};
        }
        return {pages + (size_t)(d / kTile) * tile_bytes, nullptr, (int)(d % kTile)};
    }
};

struct ToContext {
    Layout L;
    const int32_t* requests;
    const int32_t* positions;
    int tokens;
    size_t tile_bytes;
    __device__ __forceinline__ Place operator()(int64_t i, bool first) const {
        const int32_t p = __ldg(positions + i);
        const int64_t b = requests ? (int64_t)__ldg(requests + i) : i;
        if (p < 0 || b < 0) return {nullptr, nullptr, -1};
        const int32_t page = p / tokens, off = p - page * tokens;
        if (b >= L.R || page >= (L.row_len ? __ldg(L.row_len + b) : L.C)) {
            if (first) atomicOr(L.status, 1u /* HS_STATUS_RANGE */);
            return {nullptr, nullptr, -1};
        }
        const int64_t row = (L.row_base ? __ldg(L.row_base + b) : b * L.C) + page;
        const int32_t s = L.pt[(size_t)b * L.C + page];
        const size_t in = (size_t)(off / kTile) * tile_bytes;
        return {const_cast<uint8_t*>(L.host) + (size_t)row * L.host_stride + in,
                s >= 0 ? L.dev + ((size_t)b * L.S + s) * L.E + in : nullptr, off % kTile};
    }
};

// A warp takes groups of 512 / D consecutive tokens of one head (blockIdx.y), kWays groups at a
// time with all their loads in flight.
template <int D, bool BF16, class Dest>
__global__ void __launch_bounds__(kThreads) write_kernel(const TokenRows in, int64_t n, const Dest dest) {
    constexpr int kBlocks = D / 16, kTok = 32 / kBlocks, kWays = 2;
    const int lane = threadIdx.x & 31, blk = lane % kBlocks, h = blockIdx.y;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32) * (kTok * kWays);
    const uint16_t* k = in.k + h * in.k_head + 16 * blk;
    const uint16_t* v = in.v + h * in.v_head + 16 * blk;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * (kTok * kWays) + lane / kBlocks; i0 < n; i0 += step) {
        uint32_t kw[kWays][8], vw[kWays][8];
        Place p[kWays];
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
            const int64_t i = i0 + w * kTok;
            p[w].row = -1;
            if (i >= n) continue;
            load_block(kw[w], k + i * in.k_token);
            load_block(vw[w], v + i * in.v_token);
            p[w] = dest(i, h == 0 && blk == 0);
        }
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
            if (p[w].row < 0) continue;
            const Block kb = quantise<BF16>(kw[w]), vb = quantise<BF16>(vw[w]);
            uint8_t* c = p[w].a + (size_t)h * (18 * D);
            store_block<D>(c, p[w].row, blk, kb);
            store_block<D>(c + 9 * D, p[w].row, blk, vb);
            if (p[w].b) {
                c = p[w].b + (size_t)h * (18 * D);
                store_block<D>(c, p[w].row, blk, kb);
                store_block<D>(c + 9 * D, p[w].row, blk, vb);
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Two codes of a byte to two halves (exact).
__device__ __forceinline__ void decode_word(uint32_t w, uint32_t (&h)[4]) {
    asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b;"
        " cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

template <bool BF16>
__device__ __forceinline__ uint4 decode8(uint32_t w, uint32_t u) {
    uint32_t h[4], r[4];
    decode_word(w, h);
    const __half2 s = __half2half2(__ushort_as_half((uint16_t)(u << 7)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), s);  // exact
        if (BF16) {
            const float2 f = __half22float2(x);
            const __nv_bfloat162 y = __floats2bfloat162_rn(f.x, f.y);  // exact
            r[i] = *reinterpret_cast<const uint32_t*>(&y);
        } else {
            r[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// A warp takes a tile of 16 tokens of one head (blockIdx.y) of a selected page, all its loads
// in flight at once. Tiles: every page of [B][n] in turn.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
read_kernel(const uint8_t* __restrict__ pages, int S, const int32_t* __restrict__ slots, int64_t ntiles, int n, int tiles,
            int heads, uint16_t* __restrict__ ko, uint16_t* __restrict__ vo, uint32_t* status) {
    constexpr int kBlocks = D / 16, kTok = 32 / kBlocks, kWays = kTile / kTok;
    const int lane = threadIdx.x & 31, blk = lane % kBlocks, h = blockIdx.y;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t x = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); x < ntiles; x += step) {
        const int64_t j = tiles == 1 ? x : x / tiles;  // page of [B][n]
        const int tile = (int)(x - j * tiles);
        const int32_t s = __ldg(slots + j);
        const bool live = s >= 0 && s < S;
        if (s >= S && status && tile == 0 && h == 0 && lane == 0) atomicOr(status, 1u /* HS_STATUS_RANGE */);
        const int64_t b = live ? j / n : 0;
        const uint8_t* c = pages + ((size_t)((b * S + (live ? s : 0)) * tiles + tile) * heads + h) * (18 * D);
        uint2 kc[kWays], vc[kWays];
        uint32_t ku[kWays], vu[kWays];
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
            const int r = w * kTok + lane / kBlocks;
            kc[w] = vc[w] = make_uint2(0, 0);
            ku[w] = vu[w] = 0;
            if (live) {
                kc[w] = __ldg(reinterpret_cast<const uint2*>(c + r * (D / 2) + 8 * blk));
                vc[w] = __ldg(reinterpret_cast<const uint2*>(c + 9 * D + r * (D / 2) + 8 * blk));
                ku[w] = __ldg(c + 8 * D + r * (D / 16) + blk);
                vu[w] = __ldg(c + 17 * D + r * (D / 16) + blk);
            }
        }
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
            const size_t at = ((size_t)(x * kTile + w * kTok + lane / kBlocks) * heads + h) * D + 16 * blk;
            reinterpret_cast<uint4*>(ko + at)[0] = decode8<BF16>(kc[w].x, ku[w]);
            reinterpret_cast<uint4*>(ko + at)[1] = decode8<BF16>(kc[w].y, ku[w]);
            reinterpret_cast<uint4*>(vo + at)[0] = decode8<BF16>(vc[w].x, vu[w]);
            reinterpret_cast<uint4*>(vo + at)[1] = decode8<BF16>(vc[w].y, vu[w]);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches `kernel` with enough CTAs for `units` warp units of each of `heads` heads, at most
// kWave of them an SM (further units in turn), allowed to begin before the kernel ahead of it
// on the stream is done (the kernels wait for that themselves).
constexpr int kWave = 16;
template <class... Params, class... Args>
cudaError_t launch(cudaStream_t stream, int64_t units, int heads, int num_sms, void (*kernel)(Params...), Args... args) {
    const int64_t ctas = (units + kThreads / 32 - 1) / (kThreads / 32), most = ((int64_t)num_sms * kWave + heads - 1) / heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas < most ? ctas : most), (unsigned)heads);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

template <class Dest>
cudaError_t write_any(cudaStream_t stream, const PageShape& ps, bool bf16, const TokenRows& rows, int64_t n, const Dest& dest,
                      int num_sms) {
    if (n == 0) return cudaSuccess;
    const int64_t units = (n + 1024 / ps.dim - 1) / (1024 / ps.dim);
#define HS_WRITE(D_) \
    launch(stream, units, ps.heads, num_sms, bf16 ? write_kernel<D_, true, Dest> : write_kernel<D_, false, Dest>, rows, n, dest)
    return ps.dim == 64 ? HS_WRITE(64) : ps.dim == 128 ? HS_WRITE(128) : HS_WRITE(256);
#undef HS_WRITE
}

}  // namespace

cudaError_t launch_write_tokens(cudaStream_t stream, const PageShape& ps, bool bf16, const TokenRows& rows, int64_t n,
                                const int64_t* dest, uint8_t* pages, int64_t num_pages, uint32_t* status, int num_sms) {
    const ToPages d{dest, pages, num_pages * ps.tokens, (size_t)ps.heads * 18 * ps.dim, status};
    return write_any(stream, ps, bf16, rows, n, d, num_sms);
}

cudaError_t launch_append_tokens(const Layout& L, cudaStream_t stream, const PageShape& ps, bool bf16,
                                 const TokenRows& rows, int64_t n, const int32_t* requests, const int32_t* positions,
                                 int num_sms) {
    const ToContext d{L, requests, positions, ps.tokens, (size_t)ps.heads * 18 * ps.dim};
    return write_any(stream, ps, bf16, rows, n, d, num_sms);
}

cudaError_t launch_read_pages(cudaStream_t stream, const PageShape& ps, bool bf16, const uint8_t* pages, int B, int S,
                              const int32_t* slots, int n, void* k, void* v, uint32_t* status, int num_sms) {
    const int64_t ntiles = (int64_t)B * n * ps.tiles();
    if (ntiles == 0) return cudaSuccess;
#define HS_READ(D_)                                                                                                        \
    launch(stream, ntiles, ps.heads, num_sms, bf16 ? read_kernel<D_, true> : read_kernel<D_, false>, pages, S, slots, ntiles, \
           n, ps.tiles(), ps.heads, (uint16_t*)k, (uint16_t*)v, status)
    return ps.dim == 64 ? HS_READ(64) : ps.dim == 128 ? HS_READ(128) : HS_READ(256);
#undef HS_READ
}

}  // namespace hs
