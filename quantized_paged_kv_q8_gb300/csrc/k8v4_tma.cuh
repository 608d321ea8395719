// Inline-PTX wrappers of the TMA copies into shared memory, and the tensor maps of
// a cache's K and V rows.  Written from the PTX ISA's descriptions.
#pragma once

#include <cuda.h>

#include "k8v4_common.cuh"

namespace k8v4 {

// The maps of a cache's K codes and V rows: byte tensors (byte, head, cell, page)
// with boxes of 16 cells x 128 B, 128-byte swizzled (k8v4_decode.cu keeps those of
// the last caches); false when the driver refuses them.
bool tensor_maps_of(const CacheView& C, CUtensorMap* k, CUtensorMap* v);

namespace {

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

}  // namespace
}  // namespace k8v4
