// The 4-bit page format (include/hs.h, hs_page_shape) as the page kernels see it, and the
// interface between the C ABI (hs_api.cu) and those kernels (hs_page.cu, hs_page_attend.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hs_internal.h"

namespace hs {

// 16 tokens of one head: 18 D bytes -- K codes [16][D/2], K scales [16][D/16], then V's.
constexpr int kTile = 16;
constexpr int kTopScale = 0xE2;    // 10240: six times it, 61440, is still a finite half
constexpr int kBadScale = 0xFF;    // the scale of a block that holds a NaN or an infinity (a NaN)
constexpr int kMaxPageTokens = 256;

struct PageShape {
    int tokens, heads, dim;
    int tiles() const { return tokens / kTile; }
    size_t bytes() const { return (size_t)tokens * heads * dim / 8 * 9; }
    bool valid() const {
        return tokens >= kTile && tokens <= kMaxPageTokens && tokens % kTile == 0 && heads >= 1 && heads <= 65535 &&
               (dim == 64 || dim == 128 || dim == 256) && bytes() <= 0x7fffffffu;
    }
};

#ifdef __CUDACC__
// What a kernel reads that another may still have been writing when it was launched (a
// programmatic dependent): an ordinary load, never one through the read-only path.
template <class T>
__device__ __forceinline__ T load(const T* p) { return *p; }

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery, 1994).
struct Divisor {
    uint32_t d, m, s;
    Divisor() = default;
    explicit Divisor(uint32_t by) : d(by), m(0), s(0) {
        while ((1ull << s) < by) ++s;
        m = (uint32_t)((((1ull << s) - by) << 32) / by + 1);
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> s); }
};
#endif

// K and V rows of n tokens, 16-bit floats: row (token i, head h) starts i * token + h * head
// elements into the tensor, 16-byte aligned.
struct TokenRows {
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_token, k_head, v_token, v_head;
};

// Tokens into pages[num_pages] at the token slots dest[i] (page * tokens + offset; < 0: skipped).
cudaError_t launch_write_tokens(cudaStream_t stream, const PageShape& ps, bool bf16, const TokenRows& rows, int64_t n,
                                const int64_t* dest, uint8_t* pages, int64_t num_pages, uint32_t* status, int num_sms);
// Tokens into a context's history (and resident slots): token i is position positions[i] of
// request requests[i] (nullptr: request i).
cudaError_t launch_append_tokens(const Layout& L, cudaStream_t stream, const PageShape& ps, bool bf16,
                                 const TokenRows& rows, int64_t n, const int32_t* requests, const int32_t* positions,
                                 int num_sms);
// pages[B][S] -> k, v [B][n * tokens][heads][dim] through slots[B][n].
cudaError_t launch_read_pages(cudaStream_t stream, const PageShape& ps, bool bf16, const uint8_t* pages, int B, int S,
                              const int32_t* slots, int n, void* k, void* v, uint32_t* status, int num_sms);

struct PageAttention {
    const uint16_t* q;       // row (b, t, head) at b * q_batch + t * q_token + head * q_head
    uint16_t* o;
    float* lse;              // [B][Tq][Hq]
    const uint8_t* pages;    // [B][S][page bytes]
    const int32_t* slots;    // [B][k]
    const int32_t* sel;      // [B][k]
    const int32_t* lengths;  // [B]
    const int32_t* start;    // [B] or nullptr
    const int32_t* prefix;   // [B] or nullptr
    const float* slopes;     // [Hq] or nullptr
    uint32_t* status;        // or nullptr
    int64_t q_batch, q_token, q_head, o_batch, o_token, o_head;
    int B, S, k, H, G, Tq;   // H KV heads, G query heads to each
    int tiles;               // 16-token tiles of a page
    float scale, cap;
};
cudaError_t launch_attend_pages(cudaStream_t stream, const PageShape& ps, bool bf16, const PageAttention& a, int num_sms);

}  // namespace hs
