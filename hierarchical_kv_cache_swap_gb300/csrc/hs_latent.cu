// hs_latent.cu -- tokens written into 656-byte latent entries, rotary keys rotated on the way,
// and entries read back.
//
// A block is 128 consecutive values of a token's latent. Its scale is the smallest power of two
// s >= 2^-126 with 448 s >= max |x| (448 is E4M3's largest number), its codes are the E4M3 numbers
// nearest to x / s (ties to even). A power of two costs nothing in precision -- the codes float --
// and makes x / s and code * s exact: the value that an entry stands for is the one that the
// attention multiplies, with no second rounding. With a = max |x| = 1.f * 2^E, s is 2^(E - 8), or
// 2^(E - 7) where 1.f > 1.75 = 448 / 2^8. A block that holds an infinity or a NaN gets a NaN for
// its scale and reads back as NaN. The rotary key's pairs (a, b) become (a c - b s, a s + b c) in
// f32, rounded once to bf16.
//
// A warp takes a token at a time: a lane has 16 latent values, 8 lanes a block (its maximum by three
// shuffles), and one pair of the rotary key, so that each of a row's stretches moves in one access of
// the warp. Both kernels are bound by memory traffic, 1152 bytes of rows against 656 of an entry:
// 131072 tokens (237 MB) are written in 41.6 us (5.7 TB/s, 84 % of a copy's rate) and read in 38.1
// (6.2 TB/s, 92 %; a copy of as many bytes took 38.3). A decode step's 64 tokens take 1.8 and 1.5 us, the
// launches' own pace.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hs_latent.h"
#include "hs_launch.h"

namespace hs {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// What a kernel reads that another may still have been writing when it was launched (a
// programmatic dependent): an ordinary load, never one through the read-only path.
template <class T>
__device__ __forceinline__ T load(const T* p) { return *p; }

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t bits) {
    if (BF16) return __uint_as_float((uint32_t)bits << 16);
    return __half2float(__ushort_as_half(bits));
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{ .reg .b16 l, h; cvt.rn.satfinite.e4m3x2.f32 l, %2, %1; cvt.rn.satfinite.e4m3x2.f32 h, %4, %3; mov.b32 %0, {l, h}; }"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
// Four codes to four floats (exact).
__device__ __forceinline__ float4 values4(uint32_t w) {
    uint32_t l, h;
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }" : "=r"(l), "=r"(h) : "r"(w));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&l)), y = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return make_float4(x.x, x.y, y.x, y.y);
}

// Where a token's entry goes: one or two places, or none.
struct Place {
    uint8_t* a;  // nullptr: the token is skipped
    uint8_t* b;  // or nullptr
    bool bad;    // out of range
};

struct ToEntries {
    const int64_t* dest;
    uint8_t* entries;
    int64_t num;
    uint32_t* status;
    __device__ __forceinline__ Place operator()(int64_t i) const {
        const int64_t d = load(dest + i);
        if (d < 0 || d >= num) return {nullptr, nullptr, d >= 0};
        return {entries + d * kLatentEntry, nullptr, false};
    }
};

struct ToHistory {
    Layout L;
    const int32_t* requests;
    const int32_t* positions;
    uint32_t* status;
    __device__ __forceinline__ Place operator()(int64_t i) const {
        const int32_t p = load(positions + i);
        const int64_t b = requests ? (int64_t)load(requests + i) : i;
        if (p < 0 || b < 0) return {nullptr, nullptr, false};
        if (b >= L.R || p >= (L.row_len ? load(L.row_len + b) : L.C)) return {nullptr, nullptr, true};
        const int64_t row = (L.row_base ? load(L.row_base + b) : b * L.C) + p;
        const int32_t s = load(L.pt + (size_t)b * L.C + p);
        return {const_cast<uint8_t*>(L.host) + (size_t)row * L.host_stride, s >= 0 ? L.dev + ((size_t)b * L.S + s) * L.E : nullptr, false};
    }
};

// A warp's entry is 41 units of 16 bytes: lane l's codes are unit l, and lanes 0 to 8 bring the scales
// (one in each eighth lane) and the 32 words of rotary values (a lane a word) into units 32 to 40. In two
// stores instead of four, an entry's sectors are written whole but at its ends: 131072 tokens 41.6 us
// instead of 49.4.
__device__ __forceinline__ uint4 tail_unit(int lane, float scale, uint32_t word) {
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t s = __shfl_sync(0xffffffffu, __float_as_uint(scale), 8 * j);
        const uint32_t w = __shfl_sync(0xffffffffu, word, (4 * lane - 4 + j) & 31);
        r[j] = lane == 0 ? s : w;
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void store_entry(uint8_t* at, int lane, const uint4& codes, const uint4& tail) {
    reinterpret_cast<uint4*>(at)[lane] = codes;
    if (lane < 9) reinterpret_cast<uint4*>(at)[32 + lane] = tail;
}

// A warp takes `per` (at most 32) consecutive tokens: its lanes look up where each goes and its position
// in one load, so that the loop over them waits for nothing but the rows and the table's.
template <bool BF16, bool HALVES, class Dest>
__global__ void __launch_bounds__(kThreads) write_kernel(const LatentRows in, int64_t n, int per, const Rotation rot, const Dest dest) {
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * per;
    const int count = (int)(n - first < per ? n - first : per);  // may be negative
    Place mine{nullptr, nullptr, false};
    int32_t row_of = 0;
    if (lane < count) {
        mine = dest(first + lane);
        if (rot.table) {
            row_of = load(rot.positions + first + lane);
            if (mine.a && (row_of < 0 || row_of >= rot.rows)) mine = Place{nullptr, nullptr, true};
        }
        if (mine.bad && dest.status) atomicOr(dest.status, 1u /* HS_STATUS_RANGE */);
    }
#pragma unroll 2
    for (int k = 0; k < count; ++k) {
        uint8_t* const a_at = (uint8_t*)__shfl_sync(0xffffffffu, (unsigned long long)mine.a, k);
        uint8_t* const b_at = (uint8_t*)__shfl_sync(0xffffffffu, (unsigned long long)mine.b, k);
        const int32_t at = __shfl_sync(0xffffffffu, row_of, k);
        if (!a_at) continue;
        const int64_t i = first + k;
        const uint4* row = reinterpret_cast<const uint4*>(in.latent + i * in.latent_stride) + 2 * lane;
        const uint16_t* rope = in.rope + i * in.rope_stride;
        const uint4 w0 = load(row), w1 = load(row + 1);
        uint32_t pair;
        if (HALVES) pair = (uint32_t)load(rope + lane) | (uint32_t)load(rope + lane + 32) << 16;
        else pair = load(reinterpret_cast<const uint32_t*>(rope) + lane);
        float c = 1.f, s = 0.f;
        if (rot.table) {
            c = load(rot.table + (int64_t)at * kRope + lane);
            s = load(rot.table + (int64_t)at * kRope + 32 + lane);
        }
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        // the magnitudes' bits order like the magnitudes, infinities and NaNs above every number
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
        m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
        for (int d = 1; d < 8; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const bool bad = m >= (BF16 ? 0x7F80u : 0x7C00u);
        // the scale's biased exponent: a's own less 8, one more where its fraction is above .75
        const uint32_t a = __float_as_uint(to_float<BF16>((uint16_t)m));
        const int power = max((int)((a + 0x1FFFFFu) >> 23) - 8, 1);
        const float inv = bad ? 0.f : __uint_as_float((uint32_t)(254 - power) << 23);
        const float scale = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)power << 23);
        uint32_t codes[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            codes[j] = codes4(to_float<BF16>((uint16_t)w[2 * j]) * inv, to_float<BF16>((uint16_t)(w[2 * j] >> 16)) * inv,
                              to_float<BF16>((uint16_t)w[2 * j + 1]) * inv, to_float<BF16>((uint16_t)(w[2 * j + 1] >> 16)) * inv);
        const uint4 unit = make_uint4(codes[0], codes[1], codes[2], codes[3]);
        float2 r = make_float2(to_float<BF16>((uint16_t)pair), to_float<BF16>((uint16_t)(pair >> 16)));
        if (rot.table) r = turn(r.x, r.y, c, s);
        uint32_t word = pack<true>(r.x, r.y);
        if (HALVES) {  // dimensions lane and lane + 32 become 2 lane and 2 lane + 1
            const uint32_t x = __shfl_sync(0xffffffffu, word, 2 * lane & 31), y = __shfl_sync(0xffffffffu, word, (2 * lane + 1) & 31);
            word = lane < 16 ? (x & 0xFFFFu) | y << 16 : x >> 16 | (y & 0xFFFF0000u);
        }
        const uint4 tail = tail_unit(lane, scale, word);
        store_entry(a_at, lane, unit, tail);
        if (b_at) store_entry(b_at, lane, unit, tail);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(kThreads) read_kernel(const uint8_t* entries, int64_t S, const int32_t* slots, int64_t n, int64_t total, int per,
                                                        uint16_t* latent, uint16_t* rope, uint32_t* status) {
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * per;
    const int count = (int)(total - first < per ? total - first : per);  // may be negative
    int32_t slot = -1;
    int64_t of = 0;  // the entry's number
    if (lane < count) {
        slot = load(slots + first + lane);
        of = (first + lane) / n * S + slot;
        if (slot >= S && status) atomicOr(status, 1u /* HS_STATUS_RANGE */);
    }
#pragma unroll 2
    for (int k = 0; k < count; ++k) {
        const int64_t j = first + k, entry = __shfl_sync(0xffffffffu, of, k);
        const int32_t s = __shfl_sync(0xffffffffu, slot, k);
        uint4 c = make_uint4(0, 0, 0, 0);
        float scale = 0.f;
        uint32_t pair = 0;
        if (s >= 0 && s < S) {
            const uint8_t* at = entries + entry * kLatentEntry;
            c = load(reinterpret_cast<const uint4*>(at) + lane);
            scale = load(reinterpret_cast<const float*>(at + kLatent) + (lane >> 3));
            pair = load(reinterpret_cast<const uint32_t*>(at + kLatent + 16) + lane);
        }
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        uint32_t r[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = values4(w[k]);
            r[2 * k] = pack<BF16>(v.x * scale, v.y * scale);
            r[2 * k + 1] = pack<BF16>(v.z * scale, v.w * scale);
        }
        uint16_t* to = latent + j * kLatent + 16 * lane;
        if (WIDE) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                         "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
        } else {
            reinterpret_cast<uint4*>(to)[0] = make_uint4(r[0], r[1], r[2], r[3]);
            reinterpret_cast<uint4*>(to)[1] = make_uint4(r[4], r[5], r[6], r[7]);
        }
        reinterpret_cast<uint32_t*>(rope + j * kRope)[lane] =
            BF16 ? pair : pack<false>(to_float<true>((uint16_t)pair), to_float<true>((uint16_t)(pair >> 16)));
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// CTAs an SM that the items are shared over. 131072 tokens written: 45 us with 2, 41.6 with 4 (what is
// resident at 64 registers), 43 with 8, 48 with an item a warp; read: 40.5 with 12, 38.1 with 48.
constexpr int kWriteWave = 4, kReadWave = 48;
// Items of a warp: as many as `wave` CTAs an SM leave to each, at most one a lane.
int share(int64_t items, int num_sms, int wave) {
    const int64_t warps = (int64_t)num_sms * wave * kWarps, per = (items + warps - 1) / warps;
    return (int)(per < 32 ? per : 32);
}
dim3 grid_of(int64_t items, int per) { return dim3((unsigned)((items + (int64_t)per * kWarps - 1) / ((int64_t)per * kWarps))); }

template <class Dest>
cudaError_t write_any(cudaStream_t stream, bool bf16, const LatentRows& rows, int64_t n, const Rotation& rot, const Dest& dest, int num_sms) {
    if (n == 0) return cudaSuccess;
    const int per = share(n, num_sms, kWriteWave);
    return launch_dependent(stream, grid_of(n, per), kThreads, 0,
                  bf16 ? (rot.halves ? write_kernel<true, true, Dest> : write_kernel<true, false, Dest>)
                       : (rot.halves ? write_kernel<false, true, Dest> : write_kernel<false, false, Dest>),
                  rows, n, per, rot, dest);
}

}  // namespace

cudaError_t launch_write_latents(cudaStream_t stream, bool bf16, const LatentRows& rows, int64_t n, const Rotation& rot,
                                 const int64_t* dest, uint8_t* entries, int64_t num_entries, uint32_t* status, int num_sms) {
    return write_any(stream, bf16, rows, n, rot, ToEntries{dest, entries, num_entries, status}, num_sms);
}

cudaError_t launch_append_latents(const Layout& L, cudaStream_t stream, bool bf16, const LatentRows& rows, int64_t n,
                                  const Rotation& rot, const int32_t* requests, const int32_t* positions, int num_sms) {
    return write_any(stream, bf16, rows, n, rot, ToHistory{L, requests, positions, L.status}, num_sms);
}

cudaError_t launch_read_latents(cudaStream_t stream, bool bf16, const uint8_t* entries, int64_t S, const int32_t* slots, int64_t n,
                                int64_t total, void* latent, void* rope, uint32_t* status, int num_sms) {
    if (total == 0) return cudaSuccess;
    const bool wide = ((uintptr_t)latent & 31) == 0;
    const int per = share(total, num_sms, kReadWave);
    return launch_dependent(stream, grid_of(total, per), kThreads, 0,
                  bf16 ? (wide ? read_kernel<true, true> : read_kernel<true, false>) : (wide ? read_kernel<false, true> : read_kernel<false, false>),
                  entries, S, slots, n, total, per, (uint16_t*)latent, (uint16_t*)rope, status);
}

}  // namespace hs
