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
// are bound by memory traffic: 2 + 9/16 bytes a value. Measured over 131072 tokens of 8 heads
// of 128 (688 MB of traffic each): writing 105 us (6.55 TB/s, 98 % of a copy's rate), reading
// 103.5 us (6.64 TB/s, 99 %). A decode step's 64 tokens take 1.8 us to write and their pages
// 2.1 us to read, which is the launches' own pace. Appended to a context's histories, the
// 131072 tokens take 836 us: 181 GB/s over the host link, 94 % of a copy of the same bytes.
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

// The scale byte nearest to a / 6, a >= 0 a 16-bit float. a times the rounded sixth is off by
// 2^-23; a quotient half-way between two scales has at most eight significant bits and any
// other differs from it by 2^-12, so bringing the product to 16 bits first restores the ties.
// In the normal range the byte is then the top of the quotient's own bits (re-biased), rounded
// to three fraction bits; below it the scales are multiples of 2^-17.
__device__ __forceinline__ uint32_t scale_byte(float a) {
    const uint32_t b = (__float_as_uint(a * (1.f / 6.f)) + 0x80u) & 0xFFFFFF00u;
    const float t = __uint_as_float(b);
    const uint32_t normal = ((b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20) - ((127 - 15) << 3);
    const uint32_t u = t >= 6.103515625e-5f /* 2^-14 */ ? normal : (uint32_t)__float2int_rn(t * 131072.f /* 2^17 */);
    return min(u, (uint32_t)kTopScale);
}

// Eight values, in pairs, to eight codes (the first in the lowest bits).
__device__ __forceinline__ uint32_t codes8(const float2 (&y)[4]) {
    uint32_t r;
    asm("{ .reg .b8 a, b, c, d; cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7; mov.b32 %0, {a, b, c, d}; }"
        : "=r"(r)
        : "f"(y[0].x), "f"(y[0].y), "f"(y[1].x), "f"(y[1].y), "f"(y[2].x), "f"(y[2].y), "f"(y[3].x), "f"(y[3].y));
    return r;
}

// Eight codes with every negative zero made code 0.
__device__ __forceinline__ uint32_t one_zero(uint32_t w) {
    const uint32_t some = (w | w >> 1 | w >> 2) & 0x11111111u;  // magnitudes that are not zero
    return w & (0x77777777u | some << 3);
}

// x * inv to multiples of 2^-13, two values at a time.
__device__ __forceinline__ float2 round13(float2 x, float inv) {
    float2 y;
    asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %4}; mov.b64 c, {%5, %5}; fma.rn.f32x2 d, a, b, c;"
        " mov.b64 c, {%6, %6}; add.rn.f32x2 d, d, c; mov.b64 {%0, %1}, d; }"
        : "=f"(y.x), "=f"(y.y) : "f"(x.x), "f"(x.y), "f"(inv), "f"(1536.f), "f"(-1536.f));
    return y;
}

struct Block {
    uint32_t lo, hi;  // 16 codes
    uint32_t u;       // scale byte
};

// Sixteen 16-bit floats (w: 8 words) to a block.
template <bool BF16>
__device__ __forceinline__ Block quantise(const uint32_t (&w)[8]) {
    // the magnitudes' bits order like the magnitudes, infinities and NaNs above every number
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 7; i += 2) m = __vimax3_u16x2(m, w[i] & 0x7FFF7FFFu, w[i + 1] & 0x7FFF7FFFu);
    m = __vmaxu2(m, w[7] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    const bool bad = m >= (BF16 ? 0x7F80u : 0x7C00u);
    Block r;
    r.u = bad ? 0u : scale_byte(to_float<BF16>((uint16_t)m));
    float inv = 0.f;
    if (r.u) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale_value(r.u)));
    // x / s decides ties exactly although 1 / s is rounded: x * inv is brought to multiples of
    // 2^-13 (adding 1536 leaves 13 fraction bits), which every border between codes is. A
    // quotient on a border is off by 2^-22 relative before that and lands on it again; one that
    // is not differs from the border t s by at least one unit of x's last place, so by 2^-11
    // relative, 2^-13 at the smallest border (1/4): it stays on its side.
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = w[4 * c + i];
            y[i] = round13(make_float2(to_float<BF16>((uint16_t)x), to_float<BF16>((uint16_t)(x >> 16))), inv);
        }
        (c ? r.hi : r.lo) = one_zero(codes8(y));
    }
    if (bad) {
        r.lo = r.hi = 0;
        r.u = kBadScale;
    }
    return r;
}

__device__ __forceinline__ void load_block(uint32_t (&w)[8], const uint16_t* p) {
    const uint4 a = load(reinterpret_cast<const uint4*>(p)), b = load(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}
// The 32 bytes of a block: one store where they are 32-byte aligned (WIDE), else two. Reading
// 131072 tokens: 103.7 us against 111.3; the pages of a decode step's 64 tokens: .9 us less.
template <bool WIDE>
__device__ __forceinline__ void store_values(uint16_t* p, const uint4& a, const uint4& b) {
    if (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                     "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = a;
        reinterpret_cast<uint4*>(p)[1] = b;
    }
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
        const int64_t d = load(dest + i);
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
        const int32_t p = load(positions + i);
        const int64_t b = requests ? (int64_t)load(requests + i) : i;
        if (p < 0 || b < 0) return {nullptr, nullptr, -1};
        const int32_t page = p / tokens, off = p - page * tokens;
        if (b >= L.R || page >= (L.row_len ? load(L.row_len + b) : L.C)) {
            if (first) atomicOr(L.status, 1u /* HS_STATUS_RANGE */);
            return {nullptr, nullptr, -1};
        }
        const int64_t row = (L.row_base ? load(L.row_base + b) : b * L.C) + page;
        const int32_t s = L.pt[(size_t)b * L.C + page];
        const size_t in = (size_t)(off / kTile) * tile_bytes;
        return {const_cast<uint8_t*>(L.host) + (size_t)row * L.host_stride + in,
                s >= 0 ? L.dev + ((size_t)b * L.S + s) * L.E + in : nullptr, off % kTile};
    }
};

// A warp takes groups of 512 / D consecutive tokens of one head (blockIdx.y) in turn.
template <int D, bool BF16, class Dest>
__global__ void __launch_bounds__(kThreads) write_kernel(const TokenRows in, int64_t n, const Dest dest) {
    constexpr int kBlocks = D / 16, kTok = 32 / kBlocks;
    const int lane = threadIdx.x & 31, blk = lane % kBlocks, h = blockIdx.y;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32) * kTok;
    const uint16_t* k = in.k + h * in.k_head + 16 * blk;
    const uint16_t* v = in.v + h * in.v_head + 16 * blk;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kTok + lane / kBlocks; i < n; i += step) {
        uint32_t kw[8], vw[8];
        load_block(kw, k + i * in.k_token);
        load_block(vw, v + i * in.v_token);
        const Place p = dest(i, h == 0 && blk == 0);
        if (p.row < 0) continue;
        const Block kb = quantise<BF16>(kw), vb = quantise<BF16>(vw);
        uint8_t* c = p.a + (size_t)h * (18 * D);
        store_block<D>(c, p.row, blk, kb);
        store_block<D>(c + 9 * D, p.row, blk, vb);
        if (p.b) {
            c = p.b + (size_t)h * (18 * D);
            store_block<D>(c, p.row, blk, kb);
            store_block<D>(c + 9 * D, p.row, blk, vb);
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

// A warp takes 512 / D tokens of one head of a selected page. Units run over the heads first,
// so that a CTA writes whole rows of tokens: with the heads on blockIdx.y and 16 tokens a warp
// the same bytes took 139 us instead of 104 (131072 tokens, 8 heads of 128).
template <int D, bool BF16, bool WIDE>
__global__ void __launch_bounds__(kThreads)
read_kernel(const uint8_t* pages, int S, const int32_t* slots, int units, Divisor n, Divisor per_page,
            Divisor heads, uint16_t* ko, uint16_t* vo, uint32_t* status) {
    constexpr int kBlocks = D / 16, kTok = 32 / kBlocks;
    const int lane = threadIdx.x & 31, blk = lane % kBlocks, u = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (u < units) {
        const int j = per_page(u);  // page of [B][n]
        const int in = u - j * (int)per_page.d, grp = heads(in), h = in - grp * (int)heads.d;
        const int off = grp * kTok + lane / kBlocks;
        const int32_t s = load(slots + j);
        uint2 kc = make_uint2(0, 0), vc = kc;
        uint32_t ku = 0, vu = 0;
        if (s >= S) {
            if (in == 0 && lane == 0 && status) atomicOr(status, 1u /* HS_STATUS_RANGE */);
        } else if (s >= 0) {
            const int tiles = (int)per_page.d / (int)heads.d / (kTile / kTok);
            const uint8_t* c = pages + (((size_t)n(j) * S + s) * tiles + off / kTile) * heads.d * (18 * D) + (size_t)h * (18 * D);
            const int r = off % kTile;
            kc = load(reinterpret_cast<const uint2*>(c + r * (D / 2) + 8 * blk));
            vc = load(reinterpret_cast<const uint2*>(c + 9 * D + r * (D / 2) + 8 * blk));
            ku = load(c + 8 * D + r * (D / 16) + blk);
            vu = load(c + 17 * D + r * (D / 16) + blk);
        }
        const size_t at = (((size_t)j * (per_page.d / heads.d) + grp) * kTok + lane / kBlocks) * heads.d * D + (size_t)h * D + 16 * blk;
        store_values<WIDE>(ko + at, decode8<BF16>(kc.x, ku), decode8<BF16>(kc.y, ku));
        store_values<WIDE>(vo + at, decode8<BF16>(vc.x, vu), decode8<BF16>(vc.y, vu));
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches `kernel`, allowed to begin before the kernel ahead of it on the stream is done (the
// kernels wait for that themselves).
template <class... Params, class... Args>
cudaError_t launch(cudaStream_t stream, dim3 grid, void (*kernel)(Params...), Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
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
    // One group of tokens a warp, but at most kWave CTAs an SM, which then take further groups:
    // 131072 tokens, 8 heads of 128: 112.5 us with 16, 105.0 with 32, 107.6 with 128.
    constexpr int kWave = 32;
    const int64_t per = (int64_t)(kThreads / 32) * (512 / ps.dim);
    const int64_t ctas = (n + per - 1) / per, most = ((int64_t)num_sms * kWave + ps.heads - 1) / ps.heads;
    const dim3 grid((unsigned)(ctas < most ? ctas : most), (unsigned)ps.heads);
#define HS_WRITE(D_) \
    launch(stream, grid, bf16 ? write_kernel<D_, true, Dest> : write_kernel<D_, false, Dest>, rows, n, dest)
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
    const int64_t total = (int64_t)B * n;  // pages
    const int per_page = ps.tokens / (512 / ps.dim) * ps.heads;  // at most 2^23 units of a page
    const bool wide = (((uintptr_t)k | (uintptr_t)v) & 31) == 0;
    const size_t values = (size_t)ps.tokens * ps.heads * ps.dim;
    if (total == 0) return cudaSuccess;
    // 32-bit unit numbers: whole requests (or parts of one) in several launches beyond 2^30 of them
    const int64_t most = ((int64_t)1 << 30) / per_page;
    for (int64_t b = 0; b < B;) {
        const int64_t reqs = most / n > 0 ? (most / n < B - b ? most / n : B - b) : 1;
        for (int64_t j = 0; j < reqs * n;) {
            const int64_t count = reqs * n - j < most ? reqs * n - j : most;  // less than reqs * n: of one request
            const int units = (int)(count * per_page);
            const dim3 grid((unsigned)((units + kThreads / 32 - 1) / (kThreads / 32)));
            const uint8_t* from = pages + (size_t)b * S * ps.bytes();
            uint16_t *ko = (uint16_t*)k + (b * n + j) * values, *vo = (uint16_t*)v + (b * n + j) * values;
            cudaError_t e;
#define HS_READ(D_)                                                                                               \
    launch(stream, grid,                                                                                          \
           bf16 ? (wide ? read_kernel<D_, true, true> : read_kernel<D_, true, false>)                             \
                : (wide ? read_kernel<D_, false, true> : read_kernel<D_, false, false>),                          \
           from, S, slots + b * n + j, units, Divisor(n), Divisor(per_page), Divisor(ps.heads), ko, vo, status)
            e = ps.dim == 64 ? HS_READ(64) : ps.dim == 128 ? HS_READ(128) : HS_READ(256);
#undef HS_READ
            if (e != cudaSuccess) return e;
            j += count;
        }
        b += reqs;
    }
    return cudaSuccess;
}

}  // namespace hs
