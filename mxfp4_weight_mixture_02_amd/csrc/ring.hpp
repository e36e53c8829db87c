// What the tiled products share (fp8.hip, fp4.hip): direct-to-LDS copies and
// the wait for them, the order of rows in fragments and of tiles.
#pragma once

#include "common.hpp"

namespace mxmoe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// MFMA row r of a wave's W fragments is matrix row w_row(r) * F_N + fragment.
__device__ __forceinline__ int w_row(int r) { return 4 * (r & 3) + (r >> 2); }

constexpr int RAW_BUFFER_W3 = 0x00020000;   // raw buffer, untyped

// Copy from global memory to LDS: 16, 4 or 1 bytes a lane from base + off +
// soff to LDS address lds + (16, 4, 4) * lane.  As assembly, because the
// compiler makes every later LDS read wait for every such copy in flight
// that it cannot prove to go elsewhere, and with a ring of stages it can
// prove nothing.  The kernel waits itself (ring_wait) before it reads a
// stage.  A copy has no output register; its address is read at issue.  m0
// is a reserved register, which the compiler writes right before each use of
// its own: the clobber keeps such a pair on one side of a copy (none of these
// kernels has one), and its warning says only that m0 is not saved.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES>
__device__ __forceinline__ void lds_copy(u32x4 rsrc, uint32_t lds, uint32_t off, uint32_t soff) {
  if (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "m0", "memory");
  else if (BYTES == 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "m0", "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
                 ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "m0", "memory");
}
#pragma clang diagnostic pop
// Raw buffer of `bytes` bytes at p (a wave-uniform pointer).
__device__ __forceinline__ u32x4 buffer_of(const uint8_t* p, int64_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), (uint32_t)RAW_BUFFER_W3};
}

// Wait until at most `blocks` K blocks' copies of this wave are under way,
// and for all its LDS reads.
template <class T>
__device__ __forceinline__ void ring_wait(int blocks) {
  // a constant for every count that a ring of up to 4 stages has
  if (blocks <= 0)
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
  else if (blocks == 1 || T::NST <= 2)
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(T::COPIES, 0));
  else if (blocks == 2 || T::NST <= 3)
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * T::COPIES, 0));
  else
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(3 * T::COPIES, 0));
}

// Tile `item` of the order in which bands of 8 m-tiles run through all
// n-tiles, m fastest.
__device__ __forceinline__ void tile_at(int item, int ntiles, int mtiles, int& nt, int& mt) {
  const int band = item / (8 * ntiles), rows = min(8, mtiles - 8 * band);
  const int local = item - band * 8 * ntiles;
  mt = band * 8 + local % rows;
  nt = local / rows;
}

}  // namespace mxmoe
