// What the matrix products of mx.hip and xent.hip share: copies from memory
// into LDS by the buffer unit, waits for them, the order of the tiles.
#pragma once

#include <utility>

#include "device.hpp"

namespace gift {

// 16 (or 4) bytes per lane from the raw buffer (at voff) into LDS at m0 +
// 16 (4) lane.  Written in asm so that the compiler does not make every LDS
// read wait for all copies in flight: the kernel waits with explicit vmcnt
// counts.  The instruction writes no VGPR.  A copy reads M0 at the earliest
// one wait state after a scalar write of it; the compiler adds none inside asm.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rs, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(voff), "s"(rs) : "memory", "m0");
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t rs, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(lds), "v"(voff), "s"(rs) : "memory", "m0");
}
#pragma clang diagnostic pop

constexpr uint32_t kRawBufferWord3 = 0x00020000u;  // gfx9 raw buffer, 32-bit data format

// s_waitcnt immediate (gfx9: vmcnt in bits 3:0 and 15:14, expcnt 6:4,
// lgkmcnt 11:8), lgkmcnt 0
constexpr int wait_vm_lgkm0(int vm) { return (vm & 15) | 0x70 | (vm >> 4) << 14; }

__device__ __forceinline__ uint64_t uniform64(uint64_t x) {
  return ((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(x >> 32)) << 32) |
         (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)x);
}

// Tile of a workgroup: workgroups go to the XCDs in turn, so XCD x takes the
// x-th contiguous run of the tiles in an order that walks bands of kBand tile
// rows column by column: the tiles running together on one XCD (64 of 128 x
// 256: 8 x 8; 32 of 256 x 256: 4 x 8) share operand panels in its L2.
template <int kBand = 8>
__device__ __forceinline__ void tile_of(int id, int tm, int tn, int& ti, int& tj) {
  const int n = tm * tn, q = n / kXcd, rem = n % kXcd, x = id % kXcd;
  const int u = x * q + (x < rem ? x : rem) + id / kXcd;
  const int band = u / (kBand * tn), first = band * kBand;
  const int h = tm - first < kBand ? tm - first : kBand;
  const int v = u - first * tn;
  ti = first + v % h;
  tj = v / h;
}

__device__ __forceinline__ uint32_t bf16_bits(float x) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}

template <class F, int... I>
__device__ __forceinline__ void static_for_seq(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(0), ..., f(N - 1) with the index as a constant
template <int N, class F>
__device__ __forceinline__ void static_for(F f) {
  static_for_seq(f, std::make_integer_sequence<int, N>{});
}

}  // namespace gift
