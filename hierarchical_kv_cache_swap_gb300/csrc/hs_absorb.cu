// hs_absorb.cu -- the two products that put latent attention into its absorbed form. A head's key is
// U c (128 x 512 times the latent c) beside the rotary key, so <q, U c> = <U^T q, c>: the queries take
// U over once (hs_absorb_queries, which rotates their other 64 values on the way into the rows that
// hs_attend reads), and what hs_attend gives, a sum of latents, becomes the head's output by W
// (hs_expand_outputs).
//
// Both are a batch of products over the heads, [tokens x 128][128 x 512] and [tokens x 512][512 x 128],
// with the few tokens of a decode step: memory traffic bounds them, the matrices (128 KB a head each)
// at few tokens, the rows at many. So a CTA keeps a piece of a head's matrix in shared memory and takes
// tiles of tokens in turn; the products are mma.sync m16n8k16 in bf16 with f32 sums, at well under
// what the tensor cores give even in this form.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hs_latent.h"
#include "hs_launch.h"
#include "hs_once.h"

namespace hs {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAbsorbCols = 128;  // latent dimensions of a CTA

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}
// Byte offset of 16-byte unit u of row r in rows of UNITS units (a multiple of 8): eight rows' units
// lie in different banks.
template <int UNITS>
__device__ __forceinline__ uint32_t at(int r, int u) { return (uint32_t)(r * UNITS + (u ^ (r & 7))) * 16; }

// The rows [TM][units of 16 bytes] staged in shared memory to rows of `out`, `pitch` elements apart.
template <int TM, int UNITS>
__device__ __forceinline__ void store_rows(const uint8_t* from, uint16_t* out, int64_t pitch, int64_t rows) {
    for (int i = threadIdx.x; i < TM * UNITS; i += kThreads) {
        const int r = i / UNITS, u = i % UNITS;
        if (r < rows) reinterpret_cast<uint4*>(out + r * pitch)[u] = *reinterpret_cast<const uint4*>(from + at<UNITS>(r, u));
    }
}

// Grid: 4 pieces of 128 latent dimensions and one of the rotary values, the heads, shares of the tokens.
// A CTA takes tiles of TM tokens; its warps are TM / 32 (at least one) by the rest over the dimensions.
template <int TM>
__global__ void __launch_bounds__(kThreads) absorb_kernel(const HeadProduct p, const Rotation rot, uint32_t* status) {
    constexpr int kM = TM >= 32 ? 2 : 1;                     // m16 tiles of a warp
    constexpr int kWarpRows = TM / (16 * kM), kWarpCols = kWarps / kWarpRows, kN = kAbsorbCols / 8 / kWarpCols;  // n8 tiles of a warp
    static_assert(kN % 2 == 0, "two n8 tiles to a load");
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *const w = smem, *const x = smem + kHeadDim * kAbsorbCols * 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, piece = blockIdx.x, h = blockIdx.y;
    constexpr int kWidth = kHeadDim + kRope;
    const uint16_t* in = (const uint16_t*)p.x + h * p.x_head;
    uint16_t* out = p.out + (int64_t)h * (kLatent + kRope);
    const int64_t pitch = (int64_t)p.heads * (kLatent + kRope);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (piece == kLatent / kAbsorbCols) {  // a warp a token, a lane a pair
        const int first = rot.halves ? lane : 2 * lane, second = rot.halves ? lane + 32 : 2 * lane + 1;
        for (int64_t t = (int64_t)blockIdx.z * kWarps + warp; t < p.n; t += (int64_t)gridDim.z * kWarps) {
            const uint16_t* r = in + t * p.x_token + kHeadDim;
            float2 v = make_float2(__uint_as_float((uint32_t)r[first] << 16), __uint_as_float((uint32_t)r[second] << 16));
            if (rot.table) {
                const int32_t pos = rot.positions[t];
                if (pos >= 0 && pos < rot.rows) {
                    v = turn(v.x, v.y, rot.table[(int64_t)pos * kRope + lane], rot.table[(int64_t)pos * kRope + 32 + lane]);
                } else {
                    if (pos >= 0 && lane == 0 && h == 0 && status) atomicOr(status, 1u /* HS_STATUS_RANGE */);
                    v = make_float2(0.f, 0.f);
                }
            }
            uint16_t* o = out + t * pitch + kLatent;
            const uint32_t both = pack(v.x, v.y);
            if (rot.halves) {
                o[first] = (uint16_t)both;
                o[second] = (uint16_t)(both >> 16);
            } else {
                reinterpret_cast<uint32_t*>(o)[lane] = both;
            }
        }
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        return;
    }
    static_assert(kWidth == 192, "row of a query");
    for (int i = tid; i < kHeadDim * 16; i += kThreads) {
        const int d = i >> 4, u = i & 15;
        copy16(su32(w) + at<16>(d, u), p.w + h * p.w_head + d * p.w_row + piece * kAbsorbCols + 8 * u, true);
    }
    const int wr = warp / kWarpCols, wc = warp % kWarpCols;
    for (int64_t t0 = (int64_t)blockIdx.z * TM; t0 < p.n; t0 += (int64_t)gridDim.z * TM) {
        for (int i = tid; i < TM * 16; i += kThreads) {
            const int t = i >> 4, u = i & 15;
            const bool there = t0 + t < p.n;
            copy16(su32(x) + at<16>(t, u), in + (there ? t0 + t : 0) * p.x_token + 8 * u, there);
        }
        copies_landed();
        __syncthreads();
        float acc[kM][kN][4] = {};
#pragma unroll
        for (int k = 0; k < kHeadDim / 16; ++k) {
            uint32_t a[kM][4];
#pragma unroll
            for (int m = 0; m < kM; ++m) ldsm(a[m], su32(x) + at<16>((wr * kM + m) * 16 + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
            for (int n = 0; n < kN; n += 2) {
                uint32_t b[4];
                ldsm_t(b, su32(w) + at<16>(16 * k + (lane & 15), wc * kN + n + (lane >> 4)));
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    mma(acc[m][n], a[m], b[0], b[1]);
                    mma(acc[m][n + 1], a[m], b[2], b[3]);
                }
            }
        }
        __syncthreads();  // the tokens' shared memory becomes the staging of the result
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    *reinterpret_cast<uint32_t*>(x + at<16>((wr * kM + m) * 16 + 8 * r + (lane >> 2), wc * kN + n) + 4 * (lane & 3)) =
                        pack(acc[m][n][2 * r], acc[m][n][2 * r + 1]);
        __syncthreads();
        store_rows<TM, 16>(x, out + t0 * pitch + piece * kAbsorbCols, pitch, p.n - t0);
        __syncthreads();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <int TM>
constexpr uint32_t absorb_smem() { return kHeadDim * kAbsorbCols * 2 + TM * kAbsorbCols * 2; }

// Grid: pieces of TE output dimensions, the heads, shares of the tokens. The f32 rows are rounded to
// bf16 for the product, as the sums behind them have been: a relative 2^-9 of each, under the result's
// own rounding once 512 of them are summed.
template <int TM, int TE>
__global__ void __launch_bounds__(kThreads) expand_kernel(const HeadProduct p) {
    constexpr int kM = TM >= 32 ? 2 : 1, kWarpRows = TM / (16 * kM), kN = TE >= 128 ? 4 : 2;
    constexpr int kWarpCols = TE / (8 * kN), kShares = kWarps / (kWarpRows * kWarpCols);  // of the 512 dimensions
    constexpr int kUnits = kLatent / 8, kSteps = kLatent / 16 / kShares;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *const w = smem, *const x = smem + TE * kLatent * 2;
    float* const sums = reinterpret_cast<float*>(x + TM * kLatent * 2);  // [kShares - 1][TM][TE]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, e0 = blockIdx.x * TE, h = blockIdx.y;
    const float* in = (const float*)p.x + h * p.x_head;
    const int64_t pitch = (int64_t)p.heads * kHeadDim;
    uint16_t* out = p.out + (int64_t)h * kHeadDim + e0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = tid; i < TE * kUnits; i += kThreads) {
        const int e = i / kUnits, u = i % kUnits;
        copy16(su32(w) + at<kUnits>(e, u), p.w + h * p.w_head + (e0 + e) * p.w_row + 8 * u, true);
    }
    const int share = warp / (kWarpRows * kWarpCols), wr = warp / kWarpCols % kWarpRows, wc = warp % kWarpCols;
    for (int64_t t0 = (int64_t)blockIdx.z * TM; t0 < p.n; t0 += (int64_t)gridDim.z * TM) {
        for (int i = tid; i < TM * kUnits; i += kThreads) {
            const int t = i / kUnits, u = i % kUnits;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            if (t0 + t < p.n) {
                const float4* r = reinterpret_cast<const float4*>(in + (t0 + t) * p.x_token) + 2 * u;
                a = r[0];
                b = r[1];
            }
            *reinterpret_cast<uint4*>(x + at<kUnits>(t, u)) = make_uint4(pack(a.x, a.y), pack(a.z, a.w), pack(b.x, b.y), pack(b.z, b.w));
        }
        copies_landed();
        __syncthreads();
        float acc[kM][kN][4] = {};
#pragma unroll 4
        for (int k = share * kSteps; k < (share + 1) * kSteps; ++k) {
            uint32_t a[kM][4];
#pragma unroll
            for (int m = 0; m < kM; ++m) ldsm(a[m], su32(x) + at<kUnits>((wr * kM + m) * 16 + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
            for (int n = 0; n < kN; n += 2) {
                uint32_t b[4];  // 16 output dimensions by 16 latent ones
                ldsm(b, su32(w) + at<kUnits>((wc * kN + n) * 8 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    mma(acc[m][n], a[m], b[0], b[1]);
                    mma(acc[m][n + 1], a[m], b[2], b[3]);
                }
            }
        }
        auto place = [&](int m, int n, int r) { return ((wr * kM + m) * 16 + 8 * r + (lane >> 2)) * TE + (wc * kN + n) * 8 + 2 * (lane & 3); };
        if (kShares > 1) {
            if (share > 0)
                for (int m = 0; m < kM; ++m)
                    for (int n = 0; n < kN; ++n)
                        for (int r = 0; r < 2; ++r)
                            *reinterpret_cast<float2*>(sums + (share - 1) * TM * TE + place(m, n, r)) = make_float2(acc[m][n][2 * r], acc[m][n][2 * r + 1]);
            __syncthreads();
            if (share == 0)
                for (int s = 0; s < kShares - 1; ++s)
#pragma unroll
                    for (int m = 0; m < kM; ++m)
#pragma unroll
                        for (int n = 0; n < kN; ++n)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float2 v = *reinterpret_cast<const float2*>(sums + s * TM * TE + place(m, n, r));
                                acc[m][n][2 * r] += v.x;
                                acc[m][n][2 * r + 1] += v.y;
                            }
        } else {
            __syncthreads();
        }
        if (share == 0) {  // the tokens' shared memory becomes the staging of the result
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        *reinterpret_cast<uint32_t*>(x + ((wr * kM + m) * 16 + 8 * r + (lane >> 2)) * (TE * 2) + ((wc * kN + n) * 8 + 2 * (lane & 3)) * 2) =
                            pack(acc[m][n][2 * r], acc[m][n][2 * r + 1]);
        }
        __syncthreads();
        constexpr int kOut = TE / 8;
        for (int i = tid; i < TM * kOut; i += kThreads)
            if (t0 + i / kOut < p.n)
                reinterpret_cast<uint4*>(out + (t0 + i / kOut) * pitch)[i % kOut] = reinterpret_cast<const uint4*>(x)[i];
        __syncthreads();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <int TM, int TE>
constexpr uint32_t expand_smem() {
    constexpr int kM = TM >= 32 ? 2 : 1, kN = TE >= 128 ? 4 : 2, shares = kWarps / (TM / (16 * kM) * (TE / (8 * kN)));
    return TE * kLatent * 2 + TM * kLatent * 2 + (shares - 1) * TM * TE * 4;
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
        if (x == cudaSuccess) x = allow(expand_kernel<16, 32>, expand_smem<16, 32>());
        if (x == cudaSuccess) x = allow(expand_kernel<64, 128>, expand_smem<64, 128>());
        return (int)x;
    }, &ready);
}

unsigned tiles(int64_t n, int of) { return (unsigned)((n + of - 1) / of < 1024 ? (n + of - 1) / of : 1024); }

}  // namespace

cudaError_t launch_absorb_queries(cudaStream_t stream, const HeadProduct& p, const Rotation& rot, uint32_t* status, int num_sms) {
    if (p.n == 0 || p.heads == 0) return cudaSuccess;
    cudaError_t e = set_up();
    if (e != cudaSuccess) return e;
    constexpr unsigned pieces = kLatent / kAbsorbCols + 1;
    if (p.n <= 16) return launch_dependent(stream, dim3(pieces, p.heads, tiles(p.n, 16)), kThreads, absorb_smem<16>(), absorb_kernel<16>, p, rot, status);
    return launch_dependent(stream, dim3(pieces, p.heads, tiles(p.n, 64)), kThreads, absorb_smem<64>(), absorb_kernel<64>, p, rot, status);
}

cudaError_t launch_expand_outputs(cudaStream_t stream, const HeadProduct& p, int num_sms) {
    if (p.n == 0 || p.heads == 0) return cudaSuccess;
    cudaError_t e = set_up();
    if (e != cudaSuccess) return e;
    if (p.n <= 16) return launch_dependent(stream, dim3(kHeadDim / 32, p.heads, tiles(p.n, 16)), kThreads, expand_smem<16, 32>(), expand_kernel<16, 32>, p);
    return launch_dependent(stream, dim3(kHeadDim / 128, p.heads, tiles(p.n, 64)), kThreads, expand_smem<64, 128>(), expand_kernel<64, 128>, p);
}

}  // namespace hs
