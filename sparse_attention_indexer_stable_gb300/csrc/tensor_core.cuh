// tensor_core.cuh -- the fifth-generation tensor cores' instructions as the
// kernels use them: tensor memory, matrix products, tensor copies, and waits
// that end.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bulk_copy.cuh"

namespace dcp {

// ------------------------------------------------------------ tensor memory
// One warp allocates columns (a power of two, 32 to 512) and frees them.
__device__ __forceinline__ void tmem_allocate(uint32_t* dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(columns)
               : "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

#define DCP_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define DCP_R16(r, i) DCP_R4(r, i), DCP_R4(r, i + 4), DCP_R4(r, i + 8), DCP_R4(r, i + 12)
#define DCP_S4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
#define DCP_S16(r, i) DCP_S4(r, i), DCP_S4(r, i + 4), DCP_S4(r, i + 8), DCP_S4(r, i + 12)

// 32 columns of the warp's 32 lanes: a thread's registers are its lane's row.
// The wait is part of the instruction's text, so that nothing that uses the
// registers can be moved before it.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : DCP_R16(r, 0), DCP_R16(r, 16)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : DCP_R16(r, 0)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load64(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : DCP_R16(r, 0), DCP_R16(r, 16), DCP_R16(r, 32), DCP_R16(r, 48)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load128(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "{\n .reg .b32 a, b;\n mov.b32 a, %128;\n add.u32 b, %128, 64;\n"
      " tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, "
      "%34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, "
      "%50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [a];\n"
      " tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
      "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, "
      "%110, %111, %112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, "
      "%124, %125, %126, %127}, [b];\n"
      " tcgen05.wait::ld.sync.aligned;\n}"
      : DCP_R16(r, 0), DCP_R16(r, 16), DCP_R16(r, 32), DCP_R16(r, 48), DCP_R16(r, 64),
        DCP_R16(r, 80), DCP_R16(r, 96), DCP_R16(r, 112)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(taddr),
      DCP_S16(r, 0), DCP_S16(r, 16)
      : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      DCP_S16(r, 0)
      : "memory");
}

// ---------------------------------------------------------- matrix products
// Descriptors of operands in shared memory in rows of 128 bytes, swizzled by
// 128 (tensor copies write them so), atoms of 8 rows one after the other.
// K along the rows: `rows` of the operand, 64 elements of K.  Elements of K
// 16 further: 32 bytes.  64 further: the next block of rows.
__device__ __forceinline__ uint64_t rows_along_k(uint32_t smem) {
  return (uint64_t)((smem & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// K down the rows: a row is one element of K and 64 of the operand's other
// dimension, whose next 64 start `next` bytes further.  16 elements of K
// further: 2048 bytes.
__device__ __forceinline__ uint64_t rows_across_k(uint32_t smem, uint32_t next) {
  return (uint64_t)((smem & 0x3FFFF) >> 4) | (uint64_t)(next >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// fp32 sums of M x N products of two fp16 (or two bf16) operands.
constexpr uint32_t kNegateA = 1u << 13;
__host__ __device__ constexpr uint32_t mma_shape(bool bf16, int m, int n, bool b_across_k) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) |
         (b_across_k ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// d (+)= a b, 16 elements of K; by one thread.
__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t shape,
                                         bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
      : "memory");
}
// The same with a in tensor memory, two elements of K a column.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t shape,
                                         bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
      : "memory");
}
// Arrives at `bar` when all of this thread's products so far are done.
__device__ __forceinline__ void mma_commit(unsigned long long* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// One lane of a warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(r));
  return r != 0;
}
// x of lane 0: a value that the compiler knows to be the same in all lanes.
template <typename T>
__device__ __forceinline__ T same_in_all(T x) {
  return __shfl_sync(0xffffffffu, x, 0);
}

// ------------------------------------------------------------ tensor copies
__device__ __forceinline__ void tensor_load_3d(void* dst, const CUtensorMap* map, int x, int y,
                                               int z, unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tensor_store_3d(const CUtensorMap* map, const void* src, int x,
                                                int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::
                   "l"(map),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// This thread's stores have read shared memory; or have been written.
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// What this thread wrote to shared memory is seen by copies and products.
__device__ __forceinline__ void async_proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// -------------------------------------------------------------------- waits
// A CTA's waits end.  The first one that takes longer than about a second sets
// `given_up` and the device's status bit; all later ones then end at once.  Slow
// work that others wait for counts `beats`, from each of which the second begins
// anew.
#ifdef DCP_DEBUG_POISON
constexpr unsigned long long kPatience = 4000000ull;  // SM clocks: about 2 ms
#else
constexpr unsigned long long kPatience = 2000000000ull;
#endif

struct Patience {
  volatile int* given_up;
  volatile int* beats;
  unsigned int* status;
};

// Whether phase `parity` of `bar` completes before the CTA gives up.
__device__ __forceinline__ bool wait_for(unsigned long long* bar, uint32_t parity,
                                         const Patience& w) {
  if (mbar_try_wait(bar, parity)) return true;
  unsigned long long t0 = clock64();
  int seen = *w.beats;
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*w.given_up) return false;
    if (clock64() - t0 > kPatience) {
      if (*w.beats == seen) break;
      t0 = clock64();
      seen = *w.beats;
    }
  }
  *w.given_up = 1;
  atomicOr(w.status, kStatusCopyTimeout);
  return false;
}

// The same for what has to be waited for even when the CTA has given up; twice
// as long, so that it is not what gives up first, as it then does too.
__device__ __forceinline__ bool outlast(unsigned long long* bar, uint32_t parity,
                                        const Patience& w) {
  if (mbar_try_wait(bar, parity)) return true;
  unsigned long long t0 = clock64();
  int seen = *w.beats;
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (clock64() - t0 > 2 * kPatience) {
      if (*w.beats == seen) break;
      t0 = clock64();
      seen = *w.beats;
    }
  }
  *w.given_up = 1;
  atomicOr(w.status, kStatusCopyTimeout);
  return false;
}

}  // namespace dcp
