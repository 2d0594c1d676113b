// Pieces of the kernels that form matrix products in tiles (la_product.hip,
// la_loss_product.hip): copies from memory into LDS, waits, and the order in
// which tiles are dealt out. Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace la {

// Raw buffer resource over a uniform base: no stride, 2 GiB of range, the
// fourth word of a 32-bit-format buffer.
constexpr int kRsrcRange = 0x7fffffff;
constexpr int kRsrcWord3 = 0x00020000;

// 16 bytes per lane from memory to 1 KiB of LDS at `to` (lane order), without
// a register between; done when the wave's vmcnt says so.
// CACHE: 0, or kNonTemporal for what is read once.
constexpr int kNonTemporal = 2;

template <int CACHE = 0>
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t from, void* to, int offset,
                                            int uniform_offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      from, (__attribute__((address_space(3))) void*)to, 16, offset, uniform_offset, 0, CACHE);
}

// All but the last PENDING of this wave's copies have landed and its reads of
// LDS are done; so are those of every wave of the workgroup after it.
template <int PENDING>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(PENDING >= 0 && PENDING < 64, "six bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(PENDING) : "memory");
}

// Orders the wave's own LDS accesses, which lanes exchange data through.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Workgroups are dealt to the 8 XCDs in turn: give each XCD consecutive tiles
// of every 256 of a stack, so that the tiles its L2 serves share operand
// rows, and each XCD the same share of every stack (sums of one stack are
// equally long).
__device__ __forceinline__ int64_t xcd_order(int64_t w, int64_t n) {
  const int64_t base = w & ~int64_t(255);
  const int part = static_cast<int>(n - base < 256 ? n - base : 256);
  const int l = static_cast<int>(w - base), x = l & 7;
  const int q = part >> 3, r = part & 7;
  return base + x * q + (x < r ? x : r) + (l >> 3);
}

// Tile t of a matrix, in bands of four tile rows taken column by column: 32
// consecutive tiles are about 4 x 8 of them.
__device__ __forceinline__ void rectangle(int t, int tiles_m, int tiles_n, int& i, int& j) {
  const int band = t / (4 * tiles_n), first = 4 * band;
  const int rows = tiles_m - first < 4 ? tiles_m - first : 4;
  const int l = t - band * 4 * tiles_n;
  i = first + l % rows;
  j = l / rows;
}

}  // namespace la
