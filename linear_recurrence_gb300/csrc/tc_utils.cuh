// Matrix products on the 5th-generation tensor cores: tiles in shared memory,
// accumulators in tensor memory (TMEM), tcgen05 instructions in PTX.
//
// A tile holds rows of 128 bf16 values in two halves of 64: half h of row r is
// the 128 bytes at h * rows * 128 + r * 128, its 16-byte pieces permuted by r % 8 (the
// 128-byte swizzle), so that neither threads that write one piece of eight
// rows nor those that write a row meet in a bank.  The tile begins on 1024 bytes.
// The same tile serves as an operand whose rows are the outer index and whose
// values are summed over ("along"), or whose rows are summed over and whose values
// are the outer index ("across").
#pragma once

#include "device_utils.cuh"

namespace sscan {

constexpr int kTcTokens = 128;  // values of a tile's row

// Byte offset of the 16-byte piece `piece` (0 .. 15) of row r in a tile of `rows` rows.
__device__ __forceinline__ unsigned tile_piece(int r, int piece, int rows) {
    return (unsigned)((piece >> 3) * rows * 128 + r * 128 + (((piece & 7) ^ (r & 7)) << 4));
}

// Operand descriptors: address, leading and stride offsets in units of 16 bytes,
// version 1, 128-byte swizzle.
__device__ __forceinline__ uint64_t tc_desc(unsigned addr, unsigned leading, unsigned stride) {
    return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)((leading >> 4) & 0x3fffu) << 16 |
           (uint64_t)((stride >> 4) & 0x3fffu) << 32 | 1ull << 46 | 2ull << 61;
}
// summed over the values of a row, 16 of them from value 16 * step on
__device__ __forceinline__ uint64_t desc_along(unsigned tile, int rows, int step) {
    return tc_desc(tile + (step >> 2) * rows * 128 + (step & 3) * 32, 16, 1024);
}
// summed over rows, 16 of them from row 16 * step on; halves are `rows` rows apart
__device__ __forceinline__ uint64_t desc_across(unsigned tile, int rows, int step) {
    return tc_desc(tile + step * 2048, rows * 128, 1024);
}
// bf16 x bf16 -> fp32, M x N outputs; whether A and B are read across their rows
__host__ __device__ constexpr uint32_t tc_kind(int m, int n, bool a_across, bool b_across) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (a_across ? 1u << 15 : 0u) | (b_across ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(m >> 4) << 24;
}

// The thread of a converged warp that issues products.  Products take their operands from
// registers that a warp has in common, so the warp runs through their issue together: one
// thread elected by the hardware, and the others wait behind it (__syncwarp) before anything else.  Without
// that wait the others' next instructions changed descriptors under products that were being issued.
__device__ __forceinline__ bool tc_elect() {
    unsigned mine = 0;
    asm volatile("{\n .reg .pred p;\n .reg .b32 r;\n elect.sync r|p, 0xffffffff;\n @p mov.u32 %0, 1;\n}\n" : "+r"(mine));
    return mine != 0;
}
// One product with K = 16, by one thread; add: to what the accumulator holds.
__device__ __forceinline__ void tc_mma(unsigned d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"(add ? 1u : 0u)
        : "memory");
}
// The same with A in tensor memory (a column holds two values of a row).
__device__ __forceinline__ void tc_mma_ts(unsigned d, unsigned a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(kind), "r"(add ? 1u : 0u)
        : "memory");
}
// An arrival on bar once all products that this thread has issued are done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(smem_addr(bar)) : "memory");
}
// Tensor memory columns, by one warp; where they begin is written to shared memory.
__device__ __forceinline__ void tc_alloc(unsigned* where, unsigned columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(where)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tc_free(unsigned at, unsigned columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(at), "r"(columns) : "memory");
}
// Order tensor memory accesses and products around a barrier between threads.
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// 16 columns of the warp's 32 lanes (lanes 32 * (warp % 4) and up), a lane each.
__device__ __forceinline__ void tc_load16(unsigned at, float (&v)[16]) {
    unsigned* r = reinterpret_cast<unsigned*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
// Wait for the loads; v, which one of them fills, passes through so that no use of it is
// moved before the wait.
__device__ __forceinline__ void tc_wait_loads(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                   "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tc_store8(unsigned at, const unsigned (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(at)
                 : "memory");
}

// One box of a 4-D tensor map into shared memory, completing on bar.
__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];\n" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_4d(const void* map, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];\n" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}
// A run of bytes into shared memory, completing on bar (16-byte aligned, a multiple of 16),
// and the same into the L2 only.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, unsigned bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}
// Shared memory to global; bulk_store_wait: this thread's stores have read theirs.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, unsigned bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
    asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;\n" ::: "memory");
}
__device__ __forceinline__ void bulk_prefetch(const void* src, unsigned bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

__device__ __forceinline__ unsigned pack_bf16(float low, float high) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(low, high);
    return *reinterpret_cast<const unsigned*>(&p);
}

}  // namespace sscan
