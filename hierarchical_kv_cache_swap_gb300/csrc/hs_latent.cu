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
// A warp takes a token: a lane has 16 latent values, 8 lanes a block (its maximum by three
// shuffles), and one pair of the rotary key, so that each of a row's stretches moves in one
// access of the warp. Both kernels are bound by memory traffic: 1152 bytes of rows against 656.
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
template <bool BF16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    if (BF16) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
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

struct Entry {  // a lane's part
    uint4 codes;
    float scale;
    uint32_t pair;  // interleaved: dimensions 2 lane, 2 lane + 1; halves: lane, lane + 32
};
template <bool HALVES>
__device__ __forceinline__ void store_entry(uint8_t* at, int lane, const Entry& e) {
    reinterpret_cast<uint4*>(at)[lane] = e.codes;
    if ((lane & 7) == 0) reinterpret_cast<float*>(at + kLatent)[lane >> 3] = e.scale;
    uint8_t* rope = at + kLatent + 16;
    if (HALVES) {
        reinterpret_cast<uint16_t*>(rope)[lane] = (uint16_t)e.pair;
        reinterpret_cast<uint16_t*>(rope)[lane + 32] = (uint16_t)(e.pair >> 16);
    } else {
        reinterpret_cast<uint32_t*>(rope)[lane] = e.pair;
    }
}

template <bool BF16, bool HALVES, class Dest>
__global__ void __launch_bounds__(kThreads) write_kernel(const LatentRows in, int64_t n, const Rotation rot, const Dest dest) {
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < n; i += (int64_t)gridDim.x * kWarps) {
        const uint4* row = reinterpret_cast<const uint4*>(in.latent + i * in.latent_stride) + 2 * lane;
        const uint16_t* rope = in.rope + i * in.rope_stride;
        const uint4 w0 = load(row), w1 = load(row + 1);
        uint32_t pair;
        if (HALVES) pair = (uint32_t)load(rope + lane) | (uint32_t)load(rope + lane + 32) << 16;
        else pair = load(reinterpret_cast<const uint32_t*>(rope) + lane);
        Place p = dest(i);
        float c = 1.f, s = 0.f;
        if (rot.table && p.a) {
            const int32_t at = load(rot.positions + i);
            if (at < 0 || at >= rot.rows) {
                p.a = nullptr;
                p.bad = true;
            } else {
                c = load(rot.table + (int64_t)at * kRope + lane);
                s = load(rot.table + (int64_t)at * kRope + 32 + lane);
            }
        }
        if (!p.a) {
            if (p.bad && lane == 0 && dest.status) atomicOr(dest.status, 1u /* HS_STATUS_RANGE */);
            continue;
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
        Entry e;
        e.scale = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)power << 23);
        uint32_t codes[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            codes[j] = codes4(to_float<BF16>((uint16_t)w[2 * j]) * inv, to_float<BF16>((uint16_t)(w[2 * j] >> 16)) * inv,
                              to_float<BF16>((uint16_t)w[2 * j + 1]) * inv, to_float<BF16>((uint16_t)(w[2 * j + 1] >> 16)) * inv);
        e.codes = make_uint4(codes[0], codes[1], codes[2], codes[3]);
        float2 r = make_float2(to_float<BF16>((uint16_t)pair), to_float<BF16>((uint16_t)(pair >> 16)));
        if (rot.table) r = turn(r.x, r.y, c, s);
        e.pair = pack<true>(r.x, r.y);
        store_entry<HALVES>(p.a, lane, e);
        if (p.b) store_entry<HALVES>(p.b, lane, e);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(kThreads) read_kernel(const uint8_t* entries, int64_t S, const int32_t* slots, int64_t n, int64_t total,
                                                        uint16_t* latent, uint16_t* rope, uint32_t* status) {
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t j = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); j < total; j += (int64_t)gridDim.x * kWarps) {
        const int32_t s = load(slots + j);
        uint4 c = make_uint4(0, 0, 0, 0);
        float scale = 0.f;
        uint32_t pair = 0;
        if (s >= S) {
            if (lane == 0 && status) atomicOr(status, 1u /* HS_STATUS_RANGE */);
        } else if (s >= 0) {
            const uint8_t* at = entries + (j / n * S + s) * kLatentEntry;
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

// A warp for each of `items`, but at most kWave CTAs an SM, which then take further ones.
dim3 grid_of(int64_t items, int num_sms) {
    constexpr int kWave = 32;
    const int64_t ctas = (items + kWarps - 1) / kWarps, most = (int64_t)num_sms * kWave;
    return dim3((unsigned)(ctas < most ? ctas : most));
}

template <class Dest>
cudaError_t write_any(cudaStream_t stream, bool bf16, const LatentRows& rows, int64_t n, const Rotation& rot, const Dest& dest, int num_sms) {
    if (n == 0) return cudaSuccess;
    return launch_dependent(stream, grid_of(n, num_sms), kThreads, 0,
                  bf16 ? (rot.halves ? write_kernel<true, true, Dest> : write_kernel<true, false, Dest>)
                       : (rot.halves ? write_kernel<false, true, Dest> : write_kernel<false, false, Dest>),
                  rows, n, rot, dest);
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
    return launch_dependent(stream, grid_of(total, num_sms), kThreads, 0,
                  bf16 ? (wide ? read_kernel<true, true> : read_kernel<true, false>) : (wide ? read_kernel<false, true> : read_kernel<false, false>),
                  entries, S, slots, n, total, (uint16_t*)latent, (uint16_t*)rope, status);
}

}  // namespace hs
