// Latent entries (include/hs.h, hs_write_latents) and what surrounds their attention: the
// interface between the C ABI (hs_api.cu) and the kernels (hs_latent.cu, hs_absorb.cu,
// hs_prompt.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hs_internal.h"

namespace hs {

constexpr int kLatent = 512;      // values of a latent
constexpr int kRope = 64;         // values of a rotary key
constexpr int kHeadDim = 128;     // of a head's expanded keys and values
constexpr int kLatentEntry = 656; // 512 codes, 4 scales, 64 bf16

// Positions as angles: row p of `table` holds 32 cosines, then 32 sines. table == nullptr:
// nothing is rotated. Pair i is dimensions 2 i and 2 i + 1, or (halves) i and i + 32.
struct Rotation {
    const float* table;
    int64_t rows;
    const int32_t* positions;
    int halves;
};

#ifdef __CUDACC__
// Two values rounded to 16-bit floats, in a word.
template <bool BF16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    if (BF16) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}
// The pair (x, y) turned by the angle whose cosine and sine are c and s.
__device__ __forceinline__ float2 turn(float x, float y, float c, float s) {
    return make_float2(fmaf(x, c, -(y * s)), fmaf(x, s, y * c));
}
#endif

// The waits of a call's kernel (hs_set_latent_waits): the limit of each, in nanoseconds, that of a wait for
// what is still in flight after one of them ran out, and (tests) whether the first copy is withheld, so that
// they run out. A copy that landed after its CTA's end would land in another's memory: the second limit is
// never short of what a copy or a product can take.
constexpr uint64_t kLatentWaitNs = 1000000000ull, kLeastDrainNs = 10000000ull;
struct Waits {
    uint64_t ns, drain;
    int stall;
};
inline Waits waits_of(uint64_t ns, bool stall) { return Waits{ns, ns > kLeastDrainNs ? ns : kLeastDrainNs, stall ? 1 : 0}; }

// Rows of n tokens, 16-bit floats, 16-byte aligned, `latent_stride` and `rope_stride` elements apart.
struct LatentRows {
    const uint16_t* latent;
    const uint16_t* rope;
    int64_t latent_stride, rope_stride;
};

// Tokens into entries[num_entries] at dest[i] (< 0: skipped).
cudaError_t launch_write_latents(cudaStream_t stream, bool bf16, const LatentRows& rows, int64_t n, const Rotation& rot,
                                 const int64_t* dest, uint8_t* entries, int64_t num_entries, uint32_t* status, int num_sms);
// Tokens into a context's history (and resident slots), token i at position positions[i] of
// request requests[i] (nullptr: request i).
cudaError_t launch_append_latents(const Layout& L, cudaStream_t stream, bool bf16, const LatentRows& rows, int64_t n,
                                  const Rotation& rot, const int32_t* requests, const int32_t* positions, int num_sms);
// entries[B][S] -> latent [B][n][512] and rope [B][n][64] through slots[B][n].
cudaError_t launch_read_latents(cudaStream_t stream, bool bf16, const uint8_t* entries, int64_t S, const int32_t* slots, int64_t n,
                                int64_t total, void* latent, void* rope, uint32_t* status, int num_sms);

// x [n][heads][width] rows times each head's matrix w[h] [128][512] (rows `w_row` apart).
struct HeadProduct {
    const void* x;
    int64_t x_token, x_head;  // elements between tokens and between heads
    const uint16_t* w;
    int64_t w_head, w_row;
    uint16_t* out;            // contiguous
    int64_t n;
    int heads;
    Waits waits;
    uint32_t* status;         // or nullptr
};
// bf16 x [n][heads][128 + 64] -> out [n][heads][512 + 64]: x[:128] w[h], then x[128:] rotated.
cudaError_t launch_absorb_queries(cudaStream_t stream, const HeadProduct& p, const Rotation& rot, int num_sms);
// f32 x [n][heads][512] -> bf16 out [n][heads][128]: x w[h]^T.
cudaError_t launch_expand_outputs(cudaStream_t stream, const HeadProduct& p, int num_sms);

// Attention of prompts over expanded keys and values: row (token, head) of q, k, v and o starts
// token * x_token + head * x_head elements in, row token of k_rope token * r_token.
struct PromptAttention {
    const uint16_t *q, *k, *k_rope, *v;
    int64_t q_token, q_head, k_token, k_head, r_token, v_token, v_head;
    uint16_t* o;
    int64_t o_token, o_head;
    float* lse;                             // [q_rows][H]
    const int32_t *q_starts, *k_starts;     // [B + 1]
    uint32_t* status;                       // or nullptr
    int64_t q_rows, k_rows;
    int B, H;
    int causal;
    float scale;
    Waits waits;
};
cudaError_t launch_attend_prompts(cudaStream_t stream, bool bf16, const PromptAttention& a);

}  // namespace hs
