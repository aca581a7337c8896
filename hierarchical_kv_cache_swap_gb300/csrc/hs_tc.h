// The fifth-generation tensor core, its copies and its barriers (sm_103a) as the latent kernels use
// them: mbarriers with bounded waits, tensor-map copies, tcgen05 products.
#pragma once

#include <cuda.h>  // CUtensorMap (the encoder is reached through the runtime's entry point)
#include <cuda_runtime.h>
#include <stdint.h>

#include "hs_internal.h"

namespace hs {

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// One lane of a converged warp, the same one each time. A warp that issues tensor instructions runs its
// loops as a whole and only issues from one lane: the operands then stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
    return one != 0;
}

// ---------------------------------------------------------------- mbarriers
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect_tx(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
// Whether the phase of `parity` is complete, now or soon (the thread sleeps for a while; a hint for how
// long made every wait slower: 844 us instead of 790 for prompts' attention of 16384 tokens, 16 heads).
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(su32(b)), "r"(parity) : "memory");
    return ok != 0;
}
// Waits for the phase of `parity` to complete. False, with *abort set, once this wait has lasted `ns`
// nanoseconds, or when another role has set *abort: a lost hand-off then ends the CTA, not the GPU. The
// time and *abort are looked at after each try (which sleeps for a while unless the phase is complete).
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, volatile int* abort, uint64_t ns) {
    if (bar_try(b, parity)) return true;
    const uint64_t by = global_ns() + ns;
    while (!bar_try(b, parity)) {
        if (*abort) return false;
        if (global_ns() > by) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
// The same wait where others may take long before they hand over: it is given up once neither of the two
// counts at `beat` has moved within `ns`.
__device__ __forceinline__ bool bar_wait_moving(uint64_t* b, uint32_t parity, volatile int* abort, uint64_t ns, volatile uint32_t* beat) {
    if (bar_try(b, parity)) return true;
    for (uint32_t seen = beat[0] + beat[1];;) {
        const uint64_t by = global_ns() + ns;
        do {
            if (bar_try(b, parity)) return true;
            if (*abort) return false;
        } while (global_ns() <= by);
        const uint32_t now = beat[0] + beat[1];
        if (now == seen) {
            *abort = 1;
            return false;
        }
        seen = now;
    }
}
// The same wait whatever *abort says: for what must land before the CTA ends.
__device__ __forceinline__ void bar_drain(uint64_t* b, uint32_t parity, uint64_t ns) {
    int ignored = 0;
    bar_wait(b, parity, &ignored, ns);
}

// ---------------------------------------------------------------- copies by tensor maps
// A map itself, a kernel's parameter, ahead of the first copy by it.
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(su32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(su32(bar)) : "memory");
}
// A box from shared memory to global (what lies outside the tensor is not written), by one thread, which
// then waits until the shared memory has been read.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, int x, int y, int z, int w, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(src) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// ---------------------------------------------------------------- tcgen05
// A shared-memory operand of rows of 128 swizzled bytes: the low word of its descriptor (where it is,
// and `lbo`, the bytes between its 64-element columns if it is read across its rows), to which bytes / 16
// may be added, and the high word (1024 bytes from eight rows to the next eight).
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr, uint32_t lbo) { return (addr >> 4 & 0x3FFFu) | lbo >> 4 << 16; }
constexpr uint32_t kDescHigh = 1024u >> 4 | 1u << 14 /* descriptor version */ | 2u << 29 /* 128-byte swizzle */;
// kind::f16: D f32, A and B of one 16-bit type, A K-major, B K- or MN-major.
__host__ __device__ constexpr uint32_t mma_idesc(bool bf16, int m, int n, int b_mn) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    asm volatile("{ .reg .pred p; .reg .b64 x, y; setp.ne.b32 p, %4, 0; mov.b64 x, {%1, %5}; mov.b64 y, {%2, %5};"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p; }"
                 ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHigh) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t id, uint32_t acc) {
    asm volatile("{ .reg .pred p; .reg .b64 y; setp.ne.b32 p, %4, 0; mov.b64 y, {%2, %5};"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p; }"
                 ::"r"(d), "r"(a_tmem), "r"(b), "r"(id), "r"(acc), "r"(kDescHigh) : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 (16) columns of the warp's 32 lanes of tensor memory, and back (r: a word a column).
__device__ __forceinline__ void tmem_load32(uint32_t* r, uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                   "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_load16(uint32_t* r, uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
                 "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                   "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
                   "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
                   "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <uint32_t COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t* at) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(at)), "r"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <uint32_t COLS>
__device__ __forceinline__ void tmem_free(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(COLS) : "memory");
}
#endif

// The driver's tensor-map encoder, looked up once through the runtime (no link against the
// driver library); nullptr where there is none.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled tensor_map_encoder() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return (EncodeTiled) nullptr;
        }
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// A tensor [rows][heads][columns of 64] of 16-bit floats, its strides in elements, in boxes of `box_rows`
// rows of `box_columns` columns of one head: a column after the other, rows of 128 swizzled bytes.
inline bool encode_columns(CUtensorMap* map, bool bf16, const uint16_t* x, int64_t rows, int columns, int64_t heads, int64_t row, int64_t head,
                           int box_rows, int box_columns) {
    const EncodeTiled enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t size[4] = {64, (cuuint64_t)rows, (cuuint64_t)columns, (cuuint64_t)heads};
    const cuuint64_t stride[3] = {(cuuint64_t)row * 2, 128, (cuuint64_t)head * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_columns, 1}, step[4] = {1, 1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<uint16_t*>(x), size, stride, box,
               step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace hs
