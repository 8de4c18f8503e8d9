// What the kernels that stream operands through LDS by direct loads share:
// buffers with range checks, the waits that count loads, and LDS addresses
// without a provenance.
#pragma once

#include "tile_common.hpp"

namespace moe {
namespace stage {

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// No memory access crosses: the order of the loads around it is what the waits count.
__device__ __forceinline__ void order() { asm volatile("" ::: "memory"); }
__device__ __forceinline__ void step_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A lane number that the compiler cannot carry from one use to the next: what
// follows from it is formed again where it is needed instead of being held in
// registers through the loop.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8*)p));
}

template <class T>
__device__ __forceinline__ T lds_read(uint32_t a) {   // (an address without a provenance: plain pointers into an array that
  return *(const __attribute__((address_space(3))) T*)(uintptr_t)(a);   // direct loads fill make the compiler wait for every load)
}

// Buffer over `bytes` bytes from p (uniform): loads take a lane offset and a
// uniform one, so a lane keeps 32 bits of address however far the loop goes;
// what lies at `bytes` or beyond reads as zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0,
                                           __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
__device__ __forceinline__ uint4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t add) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, add, 0));
}

// A group of m rows: as few tiles as hold them, evenly filled with blocks of 16.  (m may be all of 2^31 - 1: the sums are unsigned.)
__device__ __forceinline__ int row_tiles(int m, int most) {
  return static_cast<int>((static_cast<uint32_t>(m) + static_cast<uint32_t>(most) - 1u) / static_cast<uint32_t>(most));
}
__device__ __forceinline__ int tile_frags(int m, int nb) {
  return static_cast<int>(((static_cast<uint32_t>(m) + 15u) / 16u + static_cast<uint32_t>(nb) - 1u) / static_cast<uint32_t>(nb));
}

}  // namespace stage
}  // namespace moe
