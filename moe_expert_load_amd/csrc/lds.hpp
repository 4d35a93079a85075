// Operand loads straight into LDS, transposing LDS reads and the waits around
// them, shared by the matrix kernels.
#pragma once

#include "common.hpp"

namespace moonep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

// Range-checked buffer resource over [base, base + bytes): loads past the end
// return zeros (per dword), which pads ragged row/K tails with zeros.
__device__ __forceinline__ u32x4 make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return u32x4{uint32_t(b), uint32_t(b >> 32) & 0xffffu, bytes, 0x00020000u};
}

// 16 bytes per lane from global memory straight into LDS (buffer_load ...
// lds): lane l writes lds_dst + 16*l; lds_dst must be wave-uniform.  Issued
// as inline assembly so the compiler does not pair every later LDS read with
// a wait for all such loads; the kernel waits for each stage itself
// (wait_vm) before the barrier that publishes it.
__device__ __forceinline__ void load_lds16(u32x4 rsrc, const unsigned char* lds_dst,
                                           uint32_t voff, uint32_t soff) {
  // every operand but voff is wave-uniform; make that explicit (scalar regs)
  const uint32_t l =
      (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_void*)lds_dst);
  u32x4 r;
#pragma unroll
  for (int q = 0; q < 4; ++q) r[q] = (uint32_t)__builtin_amdgcn_readfirstlane((int)rsrc[q]);
  const uint32_t so = (uint32_t)__builtin_amdgcn_readfirstlane((int)soff);
  // one wait state between the scalar write of M0 and the LDS-DMA load that
  // reads it (a hazard of this GPU generation that the compiler's hazard pass
  // cannot see inside inline assembly)
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(l), "v"(voff), "s"(r), "s"(so) : "memory");
}

// Wait until at most N vector-memory operations of this wave are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Transposing LDS read: the 16 lanes of a group each name a 64-bit piece
// (4 bf16) of a 4-row x 16-column block; lane (a, c) = (i/4, i%4) receives
// column 4a + c of rows 0..3.  Used so that an operand stored [k][col] in
// LDS arrives as 8 consecutive k per lane, the MFMA layout.
__device__ __forceinline__ u32x2 lds_tr(const unsigned char* p) {
  const i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
  return __builtin_bit_cast(u32x2, v);
}

__device__ __forceinline__ bf16x8 join(u32x2 lo, u32x2 hi) {
  return __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
}

// Workgroup barrier that orders this wave's LDS accesses around it but does
// not wait for outstanding global loads (the direct-to-LDS loads of later
// stages stay in flight; each wave waits for its own with wait_vm first).
__device__ __forceinline__ void barrier_lds() { asm volatile("s_barrier" ::: "memory"); }

}  // namespace moonep
